// Beam search over decode steps: the selection of the K best of K V candidates, and the reordering of the
// beams' states.
//
// Selection, cand(k, v) = score_k + logit_kv - lse_k.  Within a beam the candidates have the order of its
// logits, so K best logits per beam are enough, and the logits are read once: the first kernel gives each
// wavefront a part of a row and keeps its K best (one per lane, sorted) and the running maximum and sum of
// exponentials; the second joins the parts of a request's K beams.  Ties go to the lowest token, then the
// lowest beam.  Exponentials are fp32, their sums, the logarithm and the candidates fp64: beams meet at
// differences far below an fp32 candidate's step.
//
// Reordering: a thread keeps its 16 bytes of all K rows of a request in registers between reading and
// writing, so the rows can be permuted in place, and a row that stays is neither read nor written.
#include <math.h>

#include "ops_internal.h"

namespace gdr {
namespace beam {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kNone = 0x7fffffff;  // index of an empty list place

// A part's result: list of K (value, token), the maximum and the sum of exp(x - maximum).
struct Part {
    double sum;
    float max;
    int pad;
};

// Parts of a row: one per wavefront of ~16 K elements, fewer elements while there are few rows.
int parts_of(int rows, int V) {
    const int most = (V + 1023) / 1024, want = (V + 16383) / 16384;
    int p = want;
    while (p < most && p < 64 && (long)rows * p < 4096) p *= 2;
    return p < 1 ? 1 : p > 64 ? 64 : p;
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void select_parts_kernel(SelectCall c, int parts, Part *__restrict__ part,
                                                                float *__restrict__ vals, int *__restrict__ toks) {
    constexpr int es = BF16 ? 2 : 4, per = 16 / es;  // elements of an aligned 16-byte group
    constexpr int groups = BF16 ? 1 : 2;             // of a lane and step
    const int lane = threadIdx.x & 63;
    const long id = (long)blockIdx.x * kWaves + (threadIdx.x >> 6);
    if (id >= (long)c.B * c.K * parts) return;
    const long row = id / parts;
    const int p = (int)(id - row * parts);
    const char *base = c.logits + row * c.row_stride * es;
    // aligned groups of the row: group j holds elements first + j per .. + per - 1, partly outside [0, V)
    // at the ends
    const int first = -(int)((reinterpret_cast<uintptr_t>(base) % 16) / es);
    const int total = (c.V - first + per - 1) / per;
    const int each = (total + parts - 1) / parts;
    const int g0 = min(p * each, total), g1 = min(g0 + each, total);

    float best = -INFINITY;  // list place `lane`
    int tok = kNone;
    float low = -INFINITY;   // the list's last place
    int low_tok = kNone;
    float m = -INFINITY;
    double sum = 0.0;
    const int K = c.K;
    for (int j0 = g0; j0 < g1; j0 += 64 * groups) {
        float x[groups * per];
        int e0[groups];
#pragma unroll
        for (int y = 0; y < groups; ++y) {
            const int j = j0 + y * 64 + lane;
            e0[y] = first + j * per;
            const char *at = base + (int64_t)e0[y] * es;
            if (j < g1 && e0[y] >= 0 && e0[y] + per <= c.V) {
                const uint4 raw = *reinterpret_cast<const uint4 *>(at);
                const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
                for (int e = 0; e < per; ++e)
                    x[y * per + e] = BF16 ? __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16)
                                          : __uint_as_float(w[e & 3]);
            } else {
#pragma unroll
                for (int e = 0; e < per; ++e) {
                    const bool in = j < g1 && e0[y] + e >= 0 && e0[y] + e < c.V;
                    x[y * per + e] = in ? load_in<BF16>(at, e) : -INFINITY;
                }
            }
        }
        // running maximum and sum of this lane
        float top = x[0];
#pragma unroll
        for (int i = 1; i < groups * per; ++i) top = fmaxf(top, x[i]);
        if (top > m) {
            if (sum != 0.0) sum *= static_cast<double>(expf(m - top));
            m = top;
        }
        if (m != -INFINITY || top != top) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < groups * per; ++i) s += __expf(x[i] - m);
            sum += static_cast<double>(s);
        } else {
            // every element -inf or NaN so far: a NaN has to reach the sum
#pragma unroll
            for (int i = 0; i < groups * per; ++i)
                if (x[i] != x[i]) sum = NAN;
        }
        // the list: tokens come in ascending order within a lane, not across lanes
        unsigned used = 0;  // elements of this lane that were taken
        for (;;) {
            float cand = -INFINITY;
            int at = kNone, which = 0;
#pragma unroll
            for (int i = 0; i < groups * per; ++i) {
                const int t = e0[i / per] + i % per;
                const bool in = t >= 0 && t < c.V && !(used >> i & 1u) && j0 + (i / per) * 64 + lane < g1;
                if (in && (x[i] > cand || (x[i] == cand && t < at))) {
                    cand = x[i];
                    at = t;
                    which = i;
                }
            }
            const bool wins = at != kNone && (cand > low || (cand == low && at < low_tok));
            const unsigned long long who = __ballot(wins);
            if (!who) break;
            const int from = __ffsll(who) - 1;
            const float cv = __shfl(cand, from, 64);
            const int ct = __shfl(at, from, 64);
            if (lane == from) used |= 1u << which;
            const bool above = best > cv || (best == cv && tok < ct);
            const int pos = __popcll(__ballot(above && lane < K));
            const float up = __shfl_up(best, 1, 64);
            const int up_tok = __shfl_up(tok, 1, 64);
            if (lane == pos) {
                best = cv;
                tok = ct;
            } else if (lane > pos) {
                best = up;
                tok = up_tok;
            }
            low = __shfl(best, K - 1, 64);
            low_tok = __shfl(tok, K - 1, 64);
        }
    }
    float M = m;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor(M, off, 64));
    if (m != M && sum != 0.0) sum *= static_cast<double>(expf(m - M));
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if (lane == 0) {
        part[id].sum = sum;
        part[id].max = M;
    }
    if (lane < K) {
        vals[id * K + lane] = best;
        toks[id * K + lane] = tok;
    }
}

// The K best of one request's candidates, one after the other: each round every thread finds its best
// candidate behind the last one taken.
__global__ __launch_bounds__(kThreads) void select_join_kernel(SelectCall c, int parts,
                                                               const Part *__restrict__ part,
                                                               const float *__restrict__ vals,
                                                               const int *__restrict__ toks) {
    __shared__ double lse[kMaxBeams], score[kMaxBeams];
    __shared__ int kind[kMaxBeams];  // 0: candidates; 1: done; 2: nothing finite
    __shared__ double wv[kWaves];
    __shared__ int wt[kWaves];
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, K = c.K;
    if (tid < K) {
        const long row = (long)b * K + tid;
        float M = -INFINITY;
        for (int p = 0; p < parts; ++p) M = fmaxf(M, part[row * parts + p].max);
        double sum = 0.0;
        for (int p = 0; p < parts; ++p) {
            const Part x = part[row * parts + p];
            // a part without a finite value adds its sum as it is: zero, or NaN
            sum += x.max == -INFINITY ? x.sum : x.sum * exp(static_cast<double>(x.max) - static_cast<double>(M));
        }
        const double l = static_cast<double>(M) + log(sum);
        const double s = static_cast<double>(c.scores[row]);
        lse[tid] = l;
        score[tid] = s;
        kind[tid] = c.done && c.done[row] ? 1 : isfinite(s) && isfinite(l) ? 0 : 2;
    }
    __syncthreads();
    const int each = parts * K, entries = K * each;
    const int short_list = min(K, c.V);
    double last = INFINITY;
    int last_at = -1;
    for (int i = 0; i < K; ++i) {
        double best = -INFINITY;
        int at = kNone;
        for (int x = tid; x < entries; x += kThreads) {
            const int k = x / each, y = x - k * each;
            double cand = -INFINITY;
            int t = kNone;
            if (kind[k] == 0) {
                const size_t z = ((size_t)b * K + k) * each + y;
                t = toks[z];
                if (t != kNone) {
                    cand = score[k] + (static_cast<double>(vals[z]) - lse[k]);
                    if (!isfinite(cand)) cand = -INFINITY;
                }
            } else if (kind[k] == 1) {
                // pad_token at the beam's score, then the other tokens from the lowest on
                if (y == 0) {
                    t = c.pad;
                    cand = isfinite(score[k]) ? score[k] : -INFINITY;
                } else if (y < short_list) {
                    t = y - 1 < c.pad ? y - 1 : y;
                }
            } else if (y < short_list) {
                t = y;
            }
            if (t == kNone) continue;
            const int flat = k * c.V + t;
            const bool behind = cand < last || (cand == last && flat > last_at);
            if (behind && (cand > best || (cand == best && flat < at))) {
                best = cand;
                at = flat;
            }
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
            const double ob = __shfl_xor(best, off, 64);
            const int oa = __shfl_xor(at, off, 64);
            if (ob > best || (ob == best && oa < at)) {
                best = ob;
                at = oa;
            }
        }
        if (lane == 0) {
            wv[tid >> 6] = best;
            wt[tid >> 6] = at;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            if (wv[w] > best || (wv[w] == best && wt[w] < at)) {
                best = wv[w];
                at = wt[w];
            }
        __syncthreads();
        last = best;
        last_at = at;
        if (tid == 0) {
            const int k = at / c.V, t = at - k * c.V;
            const size_t z = (size_t)b * K + i;
            c.out_scores[z] = static_cast<float>(best);
            c.out_tokens[z] = t;
            c.out_parents[z] = k;
            c.out_done[z] = kind[k] == 1 || t == c.eos;
        }
    }
}

// ---- reordering
template <int MAXK, bool IN_PLACE>
__global__ __launch_bounds__(kThreads) void reorder_kernel(int B, int K, int64_t row_bytes, const char *state,
                                                           const int *__restrict__ parents, char *out) {
    __shared__ int sp[kMaxBeams];
    const int64_t cols = (row_bytes / 16 + kThreads - 1) / kThreads;
    const int64_t lb = blockIdx.x / cols;  // layer and request
    const int b = (int)(lb % B);
    if (threadIdx.x < K) {
        const int p = parents[(size_t)b * K + threadIdx.x];
        sp[threadIdx.x] = p < 0 || p >= K ? (int)threadIdx.x : p;
    }
    __syncthreads();
    const int64_t col = ((blockIdx.x - lb * cols) * kThreads + threadIdx.x) * 16;
    if (col >= row_bytes) return;
    const char *src = state + lb * K * row_bytes + col;
    char *dst = out + lb * K * row_bytes + col;
    uint4 x[MAXK];
#pragma unroll
    for (int k = 0; k < MAXK; ++k)
        if (k < K && (!IN_PLACE || sp[k] != k)) x[k] = *reinterpret_cast<const uint4 *>(src + sp[k] * row_bytes);
#pragma unroll
    for (int k = 0; k < MAXK; ++k)
        if (k < K && (!IN_PLACE || sp[k] != k)) *reinterpret_cast<uint4 *>(dst + k * row_bytes) = x[k];
}

}  // namespace

size_t select_workspace_bytes(int B, int K, int V) {
    const size_t n = (size_t)B * K * parts_of(B * K, V);
    return n * sizeof(Part) + n * K * 8;
}

hipError_t launch_select(const SelectCall &c, hipStream_t stream) {
    const int parts = parts_of(c.B * c.K, c.V);
    const size_t n = (size_t)c.B * c.K * parts;
    Part *part = static_cast<Part *>(c.ws);
    float *vals = reinterpret_cast<float *>(part + n);
    int *toks = reinterpret_cast<int *>(vals + n * c.K);
    const dim3 grid((unsigned)((n + kWaves - 1) / kWaves));
    if (c.bf16) hipLaunchKernelGGL(select_parts_kernel<true>, grid, dim3(kThreads), 0, stream, c, parts, part, vals, toks);
    else hipLaunchKernelGGL(select_parts_kernel<false>, grid, dim3(kThreads), 0, stream, c, parts, part, vals, toks);
    const hipError_t rc = hipGetLastError();
    if (rc != hipSuccess) return rc;
    hipLaunchKernelGGL(select_join_kernel, dim3((unsigned)c.B), dim3(kThreads), 0, stream, c, parts, part, vals, toks);
    return hipGetLastError();
}

hipError_t launch_reorder(int L, int B, int K, int64_t row_bytes, const void *state, const int *parents, void *out,
                          hipStream_t stream) {
    const dim3 grid((unsigned)((row_bytes / 16 + kThreads - 1) / kThreads * L * B));
    const char *s = static_cast<const char *>(state);
    char *o = static_cast<char *>(out);
#define GDR_REORDER(MK)                                                                                              \
    do {                                                                                                             \
        if (s == o)                                                                                                  \
            hipLaunchKernelGGL((reorder_kernel<MK, true>), grid, dim3(kThreads), 0, stream, B, K, row_bytes, s,      \
                               parents, o);                                                                          \
        else                                                                                                         \
            hipLaunchKernelGGL((reorder_kernel<MK, false>), grid, dim3(kThreads), 0, stream, B, K, row_bytes, s,     \
                               parents, o);                                                                          \
    } while (0)
    if (K <= 4) GDR_REORDER(4);
    else if (K <= 8) GDR_REORDER(8);
    else if (K <= 16) GDR_REORDER(16);
    else GDR_REORDER(32);
#undef GDR_REORDER
    return hipGetLastError();
}

}  // namespace beam
}  // namespace gdr
