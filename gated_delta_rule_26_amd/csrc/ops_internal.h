// Internal declarations of the per-head-decay and beam-search sources (not part of the ABI).
#pragma once

#include "gdr_internal.h"
#include "gdr_ops.h"

namespace gdr {
namespace hd {

constexpr int kThreads = 256;
constexpr int kMaxWidth = 256;
constexpr int kMaxSegments = 64;  // of one sequence: the entering state is a chain over them

// A strided [sequence, token, head, channel] tensor; strides in bytes.
struct View {
    const char *p = nullptr;
    int64_t seq = 0, tok = 0, head = 0;
    int div = 1;  // query heads per head of this tensor
};

// One walk over the sequences.  All of the family's products are one form: rows a_i read a state E that
// rows b_j, c_j are written to, in walk order i, j = 0, 1, .. within a chunk,
//   out_i = oscale lambda^i E^T a_i + pscale sum_{j<=i} lambda^{i-j} (a_i . b_j) c_j
//   E'    = lambda^n E + uscale sum_j lambda^{n-j} b_j c_j^T       (n = tokens of the chunk)
// forward:  a, b, c = q, k, v        E = lambda S         out = o
// dq:       a, b, c = d_o, v, k      E = lambda S^T       out = dq
// dv:       a, b, c = k, q, d_o      E = R, reversed      out = dv   (R_t = dL/dS_t, last E' = ds0)
// dk:       a, b, c = v, d_o, q      E = R^T, reversed    out = dk
// E is fp32 [Da, Dc] with Da, Dc the widths of a and c.
struct Walk {
    View a, b, c;
    int Da = 0, Dc = 0;
    int reverse = 0;
    float oscale = 1.f, uscale = 1.f;
    char *out = nullptr;        // [tokens, Hout, Dc], the inputs' type or (out_f32) fp32
    int out_f32 = 0;
    int zero_outside = 0;       // packed: rows outside every sequence are set to zero
    const float *e0 = nullptr;  // [N, H, Da, Dc], or with e0_t [N, H, Dc, Da]; NULL: zero
    int e0_t = 0;
    int e0_decay = 0;           // E starts from lambda e0 (forward) or e0 (reversed)
    float *ef = nullptr;        // [N, H, Da, Dc] the last state: S of the forward pass, ds0 of a reversed one
    float *u = nullptr;         // segment sums, fragment order
    float *u_t = nullptr;       // and transposed, for the walk with the widths exchanged
    // dL/dg: x holds the tensor that `out` is the gradient of; chunk_e the E of every chunk, fragment order
    View x;
    float *chunk_e = nullptr;
    double *dg_part = nullptr;  // one per workgroup
};

// The batch as the kernels see it: segments of `seg` tokens (a multiple of the chunk), `units` of them at
// most (one at least per sequence), of N sequences of T tokens (packed: T in all, cu their offsets).
struct Batch {
    int N = 0, T = 0, H = 0;
    int seg = 0, units = 0;
    int per_seq = 0;           // segments of a sequence (fixed length)
    const int *cu = nullptr;   // NULL: fixed length
    const float *g = nullptr;
};

constexpr int kMaxWalks = 3;
struct WalkSet {
    Walk w[kMaxWalks];
    Batch b;
    int count = 0;
    int slices = 0;  // column slices of a walk (the widest of them)
};

// Tile shape for rows up to `wide` and `cols` columns of the state: padded row width, chunk, columns of a slice,
// and the workgroups that a compute unit holds.
struct Shape {
    int pad, chunk, cols, resident;
};
Shape shape_of(bool bf16, int wide, int cols);
// Bytes of one E in fragment order, over all slices.
size_t frag_bytes(const Shape &s, int slices);

// The segments' sums, and the walks themselves (dg: some of them with parts of dL/dg).
hipError_t launch_segment_sums(const WalkSet &s, bool bf16, const Shape &sh, hipStream_t stream);
hipError_t launch_walks(const WalkSet &s, bool bf16, const Shape &sh, bool dg, hipStream_t stream);
// dst [rows, width] (rows = tokens Hk) = sum over the G query heads of each group of src [rows, G, width], fp32.
struct GroupSum {
    const float *src;
    void *dst;
    size_t rows;
    int width;
};
hipError_t launch_group_sums(const GroupSum &k, const GroupSum &v, bool bf16, int G, hipStream_t stream);
// dg[h] = sum over walks, units, slices of part[walk * stride + (unit H + h) slices + slice].
hipError_t launch_dg_sum(const double *part, float *dg, int units, int H, int slices, int walks, size_t stride,
                         hipStream_t stream);

struct StepCall {
    int N, M, H, Dk, Dv;
    bool bf16;
    float scale;
    View q, k, v;
    const float *g;
    float *state;
    const int *slots, *parents;
    float *state_out;
    void *o;
};
hipError_t launch_step(const StepCall &c, hipStream_t stream);

}  // namespace hd

namespace beam {

constexpr int kMaxBeams = 32;

struct SelectCall {
    int B, K, V;
    bool bf16;
    const char *logits;
    int64_t row_stride;  // elements
    const float *scores;
    const uint8_t *done;
    int eos, pad;
    float *out_scores;
    int *out_tokens, *out_parents;
    uint8_t *out_done;
    void *ws;
};
size_t select_workspace_bytes(int B, int K, int V);
hipError_t launch_select(const SelectCall &c, hipStream_t stream);
hipError_t launch_reorder(int L, int B, int K, int64_t row_bytes, const void *state, const int *parents, void *out,
                          hipStream_t stream);

}  // namespace beam
}  // namespace gdr
