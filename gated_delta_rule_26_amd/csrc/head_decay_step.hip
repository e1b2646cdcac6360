// One token of linear attention with a decay per head: S' = lambda S + k v^T, o = scale S'^T q.
//
// Bound by HBM: the fp32 state is read once and written once, 8 Dk Dv bytes per sequence and head against
// 5 Dk Dv operations.  Without a prediction nothing waits for a sum over the state's rows, so a row is
// read, updated, written and added to the output in one pass, and the columns are independent: a workgroup
// takes one (sequence, head) or a slice of its columns, so that a few sequences still fill the card.
// A thread holds four columns of every RPP-th row (one 16-byte access each, rows contiguous).
//
// Measured: 256 sequences x 16 heads of 128 x 128 (541 MB) 99-103 us, 5.3-5.5 TB/s, what a copy reaches;
// 8 beams x 8 heads of 64 x 64 (2.1 MB) 4.8 us, two latencies of memory and the launch.
//
// A search's beams continue from their parents' states: reading row parents[n] here instead of moving the
// states first saves a pass over them.
#include "ops_internal.h"

namespace gdr {
namespace hd {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kUnroll = 8;  // state rows of a thread in flight

template <bool BF16, bool NT>
__global__ __launch_bounds__(kThreads) void step_kernel(StepCall c, int cols, int slices) {
    __shared__ float sk[kMaxWidth], sq[kMaxWidth];
    __shared__ f32x4 red[kThreads];
    const int tid = threadIdx.x;
    const int nh = blockIdx.x / slices, slice = blockIdx.x - nh * slices;
    const int n = nh / c.H, h = nh - n * c.H;
    const int col0 = slice * cols, width = min(cols, c.Dv - col0);
    const int tpr = width / 4, rpp = kThreads / tpr;  // threads of a row, rows of a pass
    const int r0 = tid / tpr, col = col0 + 4 * (tid - r0 * tpr);
    const bool busy = r0 < rpp;
    const size_t size = (size_t)c.Dk * c.Dv;
    constexpr int es = BF16 ? 2 : 4;

    // the row's state: number from (-1: zero), written to number `to`
    int from = n, to = n;
    bool pad = false;
    if (c.slots) {
        from = to = c.slots[n];
        pad = from < 0 || from >= c.M;
        int twice = 0;
        for (int i = tid; i < n; i += kThreads) twice |= c.slots[i] == from;
        pad |= __syncthreads_or(twice) != 0;
    } else if (c.parents) {
        from = c.parents[n];
        if (from < 0 || from >= c.M) from = -1;
    }
    char *o = static_cast<char *>(c.o) + (((size_t)n * c.H + h) * c.Dv + col0) * es;
    if (pad) {
        if (tid < width) store_out<BF16>(o, tid, 0.f);
        return;
    }
    const float *src = from < 0 ? nullptr : c.state + ((size_t)from * c.H + h) * size;
    float *dst = c.state_out + ((size_t)to * c.H + h) * size;
    if (tid < c.Dk) {
        sk[tid] = load_in<BF16>(c.k.p + n * c.k.seq + (h / c.k.div) * c.k.head, tid);
        sq[tid] = load_in<BF16>(c.q.p + n * c.q.seq + h * c.q.head, tid);
    }
    f32x4 v = {0.f, 0.f, 0.f, 0.f}, sum = v;
    if (busy) {
        const char *pv = c.v.p + n * c.v.seq + (h / c.v.div) * c.v.head + (size_t)col * es;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = load_in<BF16>(pv, r);
    }
    const float a = expf(c.g[h]);
    __syncthreads();
    if (busy) {
        for (int base = r0; base < c.Dk; base += kUnroll * rpp) {
            f32x4 s[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int row = base + i * rpp;
                s[i] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (src && row < c.Dk) s[i] = *reinterpret_cast<const f32x4 *>(src + (size_t)row * c.Dv + col);
            }
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int row = base + i * rpp;
                if (row < c.Dk) {
                    const float k = sk[row], q = sq[row];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        s[i][r] = a * s[i][r] + k * v[r];
                        sum[r] += q * s[i][r];
                    }
                    f32x4 *at = reinterpret_cast<f32x4 *>(dst + (size_t)row * c.Dv + col);
                    if constexpr (NT) __builtin_nontemporal_store(s[i], at);
                    else *at = s[i];
                }
            }
        }
        red[tid] = sum;
    }
    __syncthreads();
    if (tid < tpr) {
        for (int i = 1; i < rpp; ++i) {
            const f32x4 x = red[i * tpr + tid];
#pragma unroll
            for (int r = 0; r < 4; ++r) sum[r] += x[r];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) store_out<BF16>(o, 4 * tid + r, c.scale * sum[r]);
    }
}

}  // namespace

hipError_t launch_step(const StepCall &c, hipStream_t stream) {
    // columns of a workgroup: all of them, or a part (32 at least, 128 contiguous bytes of a row) while the
    // grid has fewer than two workgroups per compute unit
    int cols = c.Dv;
    while (cols > 32 && cols % 8 == 0 && (cols / 2) % 4 == 0 && cols / 2 >= 32 &&
           (long)c.N * c.H * ((c.Dv + cols - 1) / cols) < 512)
        cols /= 2;
    const int slices = (c.Dv + cols - 1) / cols;
    // states past the caches are not read again before they are displaced: non-temporal stores
    const bool nt = (size_t)c.N * c.H * c.Dk * c.Dv * 4 > ((size_t)128 << 20);
    const dim3 grid((unsigned)((size_t)c.N * c.H * slices));
#define GDR_STEP(BF, NTS) hipLaunchKernelGGL((step_kernel<BF, NTS>), grid, dim3(kThreads), 0, stream, c, cols, slices)
    if (c.bf16) {
        if (nt) GDR_STEP(true, true);
        else GDR_STEP(true, false);
    } else {
        if (nt) GDR_STEP(false, true);
        else GDR_STEP(false, false);
    }
#undef GDR_STEP
    return hipGetLastError();
}

}  // namespace hd
}  // namespace gdr
