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
// A wavefront's first step bounds what can enter its list from below (the K-th highest of its lanes' maxima, by
// bisection), so that few of its first 2048 elements are inserted; after it about K / step enter.  Measured: 512
// rows of 128,003 bf16 logits (131 MB) 49 us + 13 us for the join; without the lists 36 us, without the
// exponentials 41 us, without both 28 us (the loads).  4 rows of 32,000: 6.5 + 6 us, both kernels latencies.
//
// Reordering: a thread keeps its 16 bytes of all K rows of a request in registers between reading and
// writing, so the rows can be permuted in place, and a row that stays is neither read nor written.  Measured: 256
// states of 1 MiB into a second pool 71 us (about 426 MB: 5.9 TB/s; with ordinary stores and a branch at each load
// 157 us), 4 MB in place 2.9 us.
#include <math.h>

#include "ops_internal.h"

namespace gdr {
namespace beam {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kJoinThreads = 512;
constexpr int kNone = 0x7fffffff;  // index of an empty list place

// A part's result: list of K (value, token), the maximum and the sum of exp(x - maximum).
struct Part {
    double sum;
    float max;
    int pad;
};

// Parts of a row: one per wavefront of ~16 K elements, fewer elements while there are few rows.
int parts_of(int rows, int V) {
    const int most = (V + 2047) / 2048, want = (V + 16383) / 16384;
    int p = want;
    while (p < most && p < 64 && (long)rows * p < 4096) p *= 2;
    return p < 1 ? 1 : p > 64 ? 64 : p;
}

__device__ __forceinline__ float lane_float(float x, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}

// The K best (value, token) that a wavefront has met, one per lane, best first, equal values in the order of
// their arrival (which is that of their tokens).
struct BestList {
    float best = -INFINITY;  // place `lane`
    int tok = kNone;
    // the least value that enters (the same in all lanes): while a place is empty the one that init gave, then
    // the next float above the last place's
    float least = -INFINITY;

    __device__ __forceinline__ void insert(float x, int t, int K, int lane) {
        const bool above = best > x || (best == x && tok != kNone);
        const int pos = __popcll(__ballot(above));
        // the places from pos on move up by one lane
        const float up = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(best), 0x138, 0xf, 0xf, false));
        const int up_tok = __builtin_amdgcn_update_dpp(0, tok, 0x138, 0xf, 0xf, false);
        best = lane == pos ? x : lane > pos ? up : best;
        tok = lane == pos ? t : lane > pos ? up_tok : tok;
        if (__builtin_amdgcn_readlane(tok, K - 1) != kNone) {
            const int low = __builtin_amdgcn_readlane(__float_as_int(best), K - 1);
            least = __int_as_float((low & 0x7fffffff) == 0 ? 1 : low > 0 ? low + 1 : low - 1);  // (above +inf: NaN)
        }
    }
};

// A value that K lanes' values at least reach (-inf: not found): the highest 16 bits of the K-th highest, by
// bisection over the bits of the floats in ascending order.
__device__ float reached_by(float x, bool valid, int K) {
    const uint32_t bits = __float_as_uint(x);
    const uint32_t key = valid && x == x ? (bits & 0x80000000u ? ~bits : bits | 0x80000000u) : 0u;
    uint32_t at = 0;
#pragma unroll
    for (int bit = 31; bit >= 16; --bit) {
        const uint32_t probe = at | 1u << bit;
        if (__popcll(__ballot(key >= probe)) >= K) at = probe;
    }
    if (at <= 0x007fffffu) return -INFINITY;
    return __uint_as_float(at & 0x80000000u ? at & 0x7fffffffu : ~at);
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void select_parts_kernel(SelectCall c, int parts, Part *__restrict__ part,
                                                                float *__restrict__ vals, int *__restrict__ toks) {
    constexpr int es = BF16 ? 2 : 4, per = 16 / es;  // elements of an aligned 16-byte group
    constexpr int groups = 32 / per;                 // of a lane and step: 32 elements
    const int lane = threadIdx.x & 63;
    const long id = (long)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
    const int K = c.K;

    auto element = [](const uint4 &g, int e) {
        const uint32_t w = (&g.x)[BF16 ? e / 2 : e];
        return __uint_as_float(!BF16 ? w : e & 1 ? w & 0xffff0000u : w << 16);
    };
    // groups j .. of a step (lane by lane), and which of their elements there are
    auto load = [&](int j0, uint4 (&raw)[groups], unsigned &have) {
        have = 0;
#pragma unroll
        for (int y = 0; y < groups; ++y) {
            const int j = j0 + y * 64 + lane, e0 = first + j * per;
            const char *at = base + (int64_t)e0 * es;
            if (j < g1 && e0 >= 0 && e0 + per <= c.V) {
                raw[y] = *reinterpret_cast<const uint4 *>(at);
                have |= ((1u << per) - 1) << (y * per);
            } else {
                const uint32_t none = BF16 ? 0xff80ff80u : 0xff800000u;  // -inf
                uint32_t w[4] = {none, none, none, none};
#pragma unroll
                for (int e = 0; e < per; ++e)
                    if (j < g1 && e0 + e >= 0 && e0 + e < c.V) {
                        have |= 1u << (y * per + e);
                        if constexpr (BF16) {
                            const uint32_t h = reinterpret_cast<const uint16_t *>(at)[e];
                            w[e / 2] = e & 1 ? (w[e / 2] & 0xffffu) | h << 16 : (w[e / 2] & 0xffff0000u) | h;
                        } else {
                            w[e & 3] = reinterpret_cast<const uint32_t *>(at)[e];
                        }
                    }
                raw[y] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    };

    BestList list;
    float m = -INFINITY;
    double sum = 0.0;
    uint4 raw[groups], next[groups];
    unsigned have, next_have;
    load(g0, raw, have);
    for (int j0 = g0; j0 < g1; j0 += 64 * groups) {
        if (j0 + 64 * groups < g1) load(j0 + 64 * groups, next, next_have);
        // running maximum and sum of this lane
        float top = -INFINITY;
#pragma unroll
        for (int y = 0; y < groups; ++y)
#pragma unroll
            for (int e = 0; e < per; ++e) top = fmaxf(top, element(raw[y], e));
        if (top > m) {
            if (sum != 0.0) sum *= static_cast<double>(expf(m - top));
            m = top;
        }
        // (with nothing above -inf yet the differences would be NaN: only a NaN may give one)
        const float shift = m == -INFINITY ? 0.f : m;
        float s = 0.f;
#pragma unroll
        for (int y = 0; y < groups; ++y)
#pragma unroll
            for (int e = 0; e < per; ++e)
                s += __builtin_amdgcn_exp2f((element(raw[y], e) - shift) * 1.44269504f);
        sum += static_cast<double>(s);

        // the list.  At the first step a value that K lanes reach keeps out what cannot stay.
        if (j0 == g0) list.least = reached_by(top, have != 0, K);
        if (__ballot(have != 0 && top >= list.least)) {
#pragma unroll
            for (int y = 0; y < groups; ++y) {
                const int e0 = first + (j0 + y * 64 + lane) * per;
                unsigned left = (have >> (y * per)) & ((1u << per) - 1);  // elements not looked at
                for (;;) {
                    unsigned mine = 0;
#pragma unroll
                    for (int e = 0; e < per; ++e) {
                        if (element(raw[y], e) >= list.least) mine |= 1u << e;
                    }
                    mine &= left;
                    const unsigned long long who = __ballot(mine != 0);
                    if (!who) break;
                    // the lowest token among them
                    const int from = __ffsll(who) - 1;
                    const int e = __builtin_ctz(__builtin_amdgcn_readlane(mine, from));
                    float x = element(raw[y], 0);
#pragma unroll
                    for (int i = 1; i < per; ++i) x = e == i ? element(raw[y], i) : x;
                    if (lane == from) left &= ~((2u << e) - 1);
                    if (lane < from) left = 0;
                    list.insert(lane_float(x, from), __builtin_amdgcn_readlane(e0, from) + e, K, lane);
                }
            }
        }
#pragma unroll
        for (int y = 0; y < groups; ++y) raw[y] = next[y];
        have = next_have;
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
        vals[id * K + lane] = list.best;
        toks[id * K + lane] = list.tok;
    }
}

// One request's parts joined.  A wavefront per beam: the log-sum, and the beam's K best of its parts'; then
// every one of the K K candidates counts those before it, which is its place.
__global__ __launch_bounds__(kJoinThreads) void select_join_kernel(SelectCall c, int parts,
                                                               const Part *__restrict__ part,
                                                               const float *__restrict__ vals,
                                                               const int *__restrict__ toks) {
    __shared__ double cand[kMaxBeams * kMaxBeams];
    __shared__ int flat[kMaxBeams * kMaxBeams];
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, K = c.K;
    for (int k = __builtin_amdgcn_readfirstlane(tid >> 6); k < K; k += kJoinThreads / 64) {
        const long row = (long)b * K + k;
        const double score = static_cast<double>(c.scores[row]);
        const bool done = c.done && c.done[row];
        // parts: 64 at most, one a lane
        Part x;
        x.sum = 0.0;
        x.max = -INFINITY;
        if (lane < parts) x = part[row * parts + lane];
        float M = x.max;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor(M, off, 64));
        // a part without a finite value adds its sum as it is: zero, or NaN
        double sum = x.max == -INFINITY ? x.sum : x.sum * exp(static_cast<double>(x.max) - static_cast<double>(M));
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
        const double lse = static_cast<double>(M) + log(sum);
        const bool live = !done && isfinite(score) && isfinite(lse);
        double value = -INFINITY;
        int t = kNone;
        if (live) {
            BestList list;
            const float *v = vals + row * parts * K;
            const int *w = toks + row * parts * K;
            for (int x0 = 0; x0 < parts * K; x0 += 64) {
                const bool in = x0 + lane < parts * K;
                const float val = in ? v[x0 + lane] : -INFINITY;
                const int tk = in ? w[x0 + lane] : kNone;
                if (x0 == 0) list.least = reached_by(val, tk != kNone, K);
                bool left = tk != kNone;
                for (;;) {
                    const unsigned long long who = __ballot(left && val >= list.least);
                    if (!who) break;
                    const int from = __ffsll(who) - 1;
                    if (lane <= from) left = false;
                    list.insert(lane_float(val, from), __builtin_amdgcn_readlane(tk, from), K, lane);
                }
            }
            t = list.tok;
            if (t != kNone) {
                value = score + (static_cast<double>(list.best) - lse);
                if (!isfinite(value)) value = -INFINITY;
            }
        } else if (lane < c.V) {
            // nothing finite: the lowest tokens; done: pad_token at the beam's score before them
            t = lane;
            if (done) {
                t = lane == 0 ? c.pad : lane - 1 < c.pad ? lane - 1 : lane;
                if (lane == 0 && isfinite(score)) value = score;
            }
        }
        if (lane < K) {
            cand[k * K + lane] = value;
            flat[k * K + lane] = t == kNone ? kNone : k * c.V + t;
        }
    }
    __syncthreads();
    for (int i = tid; i < K * K; i += kJoinThreads) {
        const double mine = cand[i];
        const int at = flat[i];
        if (at == kNone) continue;
        int place = 0;
#pragma unroll 8
        for (int j = 0; j < K * K; ++j) {
            const double other = cand[j];
            place += other > mine || (other == mine && flat[j] < at);
        }
        if (place < K) {
            const int k = at / c.V, t = at - k * c.V;
            const size_t z = (size_t)b * K + place;
            c.out_scores[z] = static_cast<float>(mine);
            c.out_tokens[z] = t;
            c.out_parents[z] = k;
            c.out_done[z] = (c.done && c.done[(size_t)b * K + k]) || t == c.eos;
        }
    }
}

// ---- reordering
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

template <int MAXK, bool IN_PLACE, bool STREAM>
__global__ __launch_bounds__(kThreads) void reorder_kernel(int B, int K, int64_t row_bytes, int cols, const char *state,
                                                           const int *__restrict__ parents, char *out) {
    const int lb = blockIdx.x / cols;  // layer and request
    const int *p = parents + (size_t)(lb % B) * K;
    const int64_t col = ((int64_t)(blockIdx.x - lb * cols) * kThreads + threadIdx.x) * 16;
    if (col >= row_bytes) return;
    const char *src = state + lb * K * row_bytes + col;
    char *dst = out + lb * K * row_bytes + col;
    // The row that each row takes (the same in all threads).  In place, a row that stays loads what another one
    // does, and is not written: no branch stands between the loads.
    int from[MAXK], any = -1;
#pragma unroll
    for (int k = 0; k < MAXK; ++k) {
        from[k] = k < K ? __builtin_amdgcn_readfirstlane(p[k < K ? k : 0]) : 0;
        if (k < K && (from[k] < 0 || from[k] >= K)) from[k] = k;
        if (k < K && from[k] != k && any < 0) any = from[k];
    }
    if (IN_PLACE && any < 0) return;
    u32x4 x[MAXK];
#pragma unroll
    for (int k = 0; k < MAXK; ++k) {
        const int row = IN_PLACE && (k >= K || from[k] == k) ? any : from[k];
        x[k] = *reinterpret_cast<const u32x4 *>(src + row * row_bytes);
    }
#pragma unroll
    for (int k = 0; k < MAXK; ++k)
        if (k < K && (!IN_PLACE || from[k] != k)) {
            u32x4 *at = reinterpret_cast<u32x4 *>(dst + k * row_bytes);
            if constexpr (STREAM) __builtin_nontemporal_store(x[k], at);
            else *at = x[k];
        }
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
    hipLaunchKernelGGL(select_join_kernel, dim3((unsigned)c.B), dim3(kJoinThreads), 0, stream, c, parts, part, vals, toks);
    return hipGetLastError();
}

hipError_t launch_reorder(int L, int B, int K, int64_t row_bytes, const void *state, const int *parents, void *out,
                          hipStream_t stream) {
    const int cols = (int)((row_bytes / 16 + kThreads - 1) / kThreads);
    const dim3 grid((unsigned)((size_t)cols * L * B));
    const char *s = static_cast<const char *>(state);
    char *o = static_cast<char *>(out);
    // states past the caches are not read again before they are displaced: non-temporal stores
    const bool stream_out = (double)L * B * K * (double)row_bytes > (double)(128 << 20);
#define GDR_REORDER2(MK, IP, ST)                                                                                \
    hipLaunchKernelGGL((reorder_kernel<MK, IP, ST>), grid, dim3(kThreads), 0, stream, B, K, row_bytes, cols, s, \
                       parents, o)
#define GDR_REORDER(MK)                                    \
    do {                                                   \
        if (s == o) {                                      \
            if (stream_out) GDR_REORDER2(MK, true, true);  \
            else GDR_REORDER2(MK, true, false);            \
        } else {                                           \
            if (stream_out) GDR_REORDER2(MK, false, true); \
            else GDR_REORDER2(MK, false, false);           \
        }                                                  \
    } while (0)
    if (K <= 4) GDR_REORDER(4);
    else if (K <= 8) GDR_REORDER(8);
    else if (K <= 16) GDR_REORDER(16);
    else GDR_REORDER(32);
#undef GDR_REORDER
#undef GDR_REORDER2
    return hipGetLastError();
}

}  // namespace beam
}  // namespace gdr
