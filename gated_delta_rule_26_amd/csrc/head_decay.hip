// Linear attention with one decay per head: the chunked forward and backward passes.
//
// Every product of the family is one walk (struct Walk, ops_internal.h): with lambda = exp(g_h), walk order
// i, j = 0 .. n-1 inside a chunk, and the fp32 state E,
//   out_i = oscale lambda^i E^T a_i + pscale sum_{j<=i} lambda^{i-j} (a_i . b_j) c_j
//   E'    = lambda^n E + uscale sum_j lambda^{n-j} b_j c_j^T
// which is o (a, b, c = q, k, v), dq (d_o, v, k), and in reversed time dv (k, q, d_o) and dk (v, d_o, q).
// dL/dg = sum_t <dL/dS_t, lambda S_{t-1}> adds, over all pairs of a write and a read, the pair's value times its
// distance, which is split at the chunks' borders into parts that are each a weighted product the walks have at
// hand (no difference of large sums): (i - j) inside a chunk, i + 1 from its start, n - 1 - j to its end, and n
// for pairs across a whole chunk, lambda^n <S, R>, for which dq's walk keeps every chunk's state.
//
// Long sequences are cut into segments, so that a few heads fill the card: the first kernel sums each
// segment's writes from a zero state, U = sum_j lambda^{len-j} b_j c_j^T (the walk without outputs), and the
// walk of segment s starts from E = lambda^len E + U over the segments before it.  dk's states are dv's
// transposed: their sums are formed once and written twice.
//
// One workgroup of eight (up to 64 columns, or rows wider than 128: four) wavefronts walks one segment of one
// head and a slice of c's columns, 16 of them per wavefront, so that the state never leaves the registers: the
// 16x16 tiles of E that the update's MFMAs accumulate (rows: a's channels, columns: c's) are, lane by lane, the
// operand of the state's read, when the read's other operand is taken in the permuted order of matrix_common.h.
// The pair matrix is shared: its lower 16x16 tiles are spread over the wavefronts, which exchange them through
// LDS as operand fragments.  All outputs are formed transposed (rows: c's channels, columns: tokens), so that the
// decay of a token is a factor per lane and a lane holds consecutive channels of a token.  The rows of the next
// chunk are loaded into registers while this one is computed.
//
// Roundings below fp32 with bf16 inputs (products of bf16 values are exact in fp32): the pair matrix is rounded
// to bf16 before it meets c (2^-8 of each pair at most, of the size of the output's own rounding); the state's
// read takes it as bf16 hi + lo (2^-16): dropping lo would add an error of the output rounding's size, for 5 %
// of the time; the decayed c of the update is hi + mid + lo, 24 bits, since the state is fp32 for the caller and its
// errors would add up over the chunks.  With fp32 inputs all products are fp32 MFMAs.
//
// Measured on one MI355X (bf16, 16 heads of 128 x 128; a copy reaches 5.5 TB/s):
//   4 x 4096 tokens forward: sums 39 us + walks 85 us for 273 MB (floor 50 us).  Without its products the walk
//   takes 63 us (its loads, stores and start), without its loads 77 us: it is bound by both, the products of a
//   chunk (94 MFMAs and 340 vector instructions a wavefront, 420 KB of LDS reads in all) a little more.
//   2 x 8192 tokens backward, fixed decays: sums 83 us + three walks 187 us (floor 86 us).
// Not better: 32 columns a wavefront on four wavefronts (the same time), slices of 64 columns (the pair matrix
// twice: 108 against 91 us), more segments than the card holds at once (512 -> 768 workgroups: 118 -> 130 us), heads
// of a segment on one XCD (the same), two chunks of loads ahead in the sums (the same).  Anything that makes the
// register allocator spill inside the loop costs 15 %: a reload waits for all loads on the way.
#include <algorithm>

#include "matrix_common.h"
#include "ops_internal.h"

namespace gdr {
namespace hd {
namespace {

using mx::bf16x4;
using mx::bf16x8;
using mx::f32x4;

constexpr int kFar = 0x60000000;  // a byte offset out of any chunk's range, steps of a chunk's rows added or not

__device__ __forceinline__ float decay_power(float g, int x) { return x == 0 ? 1.f : expf(static_cast<float>(x) * g); }

// Inclusive scan over the workgroup's WV wavefronts; `tmp` holds WV values.  Two barriers.
template <bool MAX, int WV>
__device__ int block_scan(int x, int *tmp) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int y = __shfl_up(x, off, 64);
        if (lane >= off) x = MAX ? max(x, y) : x + y;
    }
    __syncthreads();
    if (lane == 63) tmp[w] = x;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WV - 1; ++i)
        if (i < w) x = MAX ? max(x, tmp[i]) : x + tmp[i];
    return x;
}

// Where segment unit u lies: sequence n (-1: none), its first token's row tok0 (0 in a fixed-length batch)
// and length, the segment's number s of ns and its tokens [t0, t0 + len) of the sequence.  first, last: the
// rows that the sequences of a packed batch cover (unit 0 only).  chunk0: the number of the segment's first
// chunk among those of all sequences, where COUNT asks for it.
struct Place {
    int n, tok0, seq_len, s, ns, t0, len, first, last, chunk0;
};

struct PlaceSmem {
    int tmp[8];
    int found[6];
};

template <int CH, bool COUNT, int WV>
__device__ Place find_place(const Batch &b, int u, PlaceSmem &sm) {
    Place p;
    p.first = 0;
    p.last = b.T;
    if (!b.cu) {
        p.n = u / b.per_seq;
        p.s = u - p.n * b.per_seq;
        p.ns = b.per_seq;
        p.tok0 = 0;
        p.seq_len = b.T;
        p.chunk0 = p.n * ((b.T + CH - 1) / CH);
    } else {
        // offsets clamped to [0, T] and raised to the largest before them; sequence i owns
        // max(1, ceil(len / seg)) units
        const int t = threadIdx.x;
        if (t == 0) sm.found[0] = -1;
        int top = 0, units = 0, chunks = 0;
        p.first = min(max(b.cu[0], 0), b.T);
        for (int base = 0; base < b.N; base += 64 * WV) {
            const int i = base + t;
            const int lo = i <= b.N ? min(max(b.cu[i], 0), b.T) : 0;
            const int hi = i < b.N ? min(max(b.cu[i + 1], 0), b.T) : 0;
            const int start = max(top, block_scan<true, WV>(lo, sm.tmp));
            const int end = max(start, hi);
            const int mine = i < b.N ? max(1, (end - start + b.seg - 1) / b.seg) : 0;
            const int upto = units + block_scan<false, WV>(mine, sm.tmp);
            const int own = i < b.N ? (end - start + CH - 1) / CH : 0;
            int chunks_to = 0;
            if constexpr (COUNT) chunks_to = chunks + block_scan<false, WV>(own, sm.tmp);
            if (i < b.N && u >= upto - mine && u < upto) {
                sm.found[0] = i;
                sm.found[1] = start;
                sm.found[2] = end - start;
                sm.found[3] = u - (upto - mine);
                sm.found[4] = mine;
                sm.found[5] = chunks_to - own;
            }
            __syncthreads();  // the scans' last reads of tmp are done
            if (t == 64 * WV - 1) {
                sm.tmp[0] = max(start, end);
                sm.tmp[1] = upto;
                sm.tmp[2] = chunks_to;
            }
            __syncthreads();
            top = sm.tmp[0];
            units = sm.tmp[1];
            chunks = sm.tmp[2];
            if (u > 0 && u < units) break;
        }
        __syncthreads();
        // the same in all lanes: kept in scalar registers
        p.last = __builtin_amdgcn_readfirstlane(top);
        p.n = __builtin_amdgcn_readfirstlane(sm.found[0]);
        p.tok0 = __builtin_amdgcn_readfirstlane(sm.found[1]);
        p.seq_len = __builtin_amdgcn_readfirstlane(sm.found[2]);
        p.s = __builtin_amdgcn_readfirstlane(sm.found[3]);
        p.ns = __builtin_amdgcn_readfirstlane(sm.found[4]);
        p.chunk0 = __builtin_amdgcn_readfirstlane(sm.found[5]);
        if (p.n < 0) return p;
    }
    p.t0 = p.s * b.seg;
    p.len = min(b.seg, p.seq_len - p.t0);
    p.chunk0 += p.t0 / CH;
    return p;
}

// ---- element types: operand fragments of `depth` terms; term e of lane group lg (lane / 16) is term
// kperm(lg, e) of a 32-block (bf16) or 4 lg + e of a 16-block (fp32).
template <bool BF16>
struct El;
template <>
struct El<true> {
    static constexpr int bytes = 2, depth = 32;
    using frag = bf16x8;
    typedef __bf16 lds;
};
template <>
struct El<false> {
    static constexpr int bytes = 4, depth = 16;
    using frag = f32x4;
    typedef float lds;
};

__device__ __forceinline__ f32x4 mul_add(bf16x8 a, bf16x8 b, f32x4 c) { return mx::mma(a, b, c); }
__device__ __forceinline__ f32x4 mul_add(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = mx::mma32(a[e], b[e], c);
    return c;
}

// ---- a tile of ROWS tokens x W channels: global -> registers -> LDS, 16 bytes a lane.  Orders of the channels
// in LDS, so that both the 16-byte accesses of rows and the transposing reads of 4x16 blocks take every bank once:
//   kRows     read by rows only.  bf16: the fragments of lane group lg, 16 bytes a row and 32-block, in a plane of
//             their own, rows an odd number of 16-byte pieces long: any 16 rows' reads take all banks, whichever
//             lane groups they are read by
//   kBoth     read by rows and transposed: as they come
//   kColumns  read transposed only: as they come
// (bf16 rows of kBoth and kColumns are 8 words longer than a multiple of the banks: the 8 rows x 32 bytes of a
// transposing read's half lie side by side.)
enum Order { kRows, kBoth, kColumns };

template <bool BF16, int W, int ROWS, Order ORD, int WV>
struct Tile {
    using T = El<BF16>;
    static constexpr int per = 16 / T::bytes;       // elements of a piece
    static constexpr int pieces = W / per;          // of a row
    static constexpr int rpp = 64 * WV / pieces;    // rows of a pass
    static constexpr int passes = ROWS / rpp;
    static constexpr int ld = W + (BF16 ? (ORD == kRows ? 8 : 16) : 4);
    static_assert(64 * WV % pieces == 0 && ROWS % rpp == 0, "tile must divide among the threads");
    // kRows of bf16: elements of a row in a plane, and of a plane (planes 2 and 3 half the banks further)
    static constexpr int prow = 8 * (W / 32 + 1), plane = ROWS * prow;
    static constexpr int size = BF16 && ORD == kRows ? 4 * plane + 64 : ROWS * ld;  // elements in LDS
    static_assert(ORD != kRows || !BF16 || (prow % 16 == 8 && plane % 128 == 0), "planes start at the same bank");
    uint4 r[passes];

    // This thread's first byte of a chunk of `stride` bytes a row, out of any chunk's range where the channel
    // is past `width`.
    static __device__ __forceinline__ int first(int stride, int col0, int width) {
        const int col = col0 + (int)(threadIdx.x % pieces) * per;
        return col < width ? (int)(threadIdx.x / pieces) * stride + col * T::bytes : kFar;
    }
    // Rows 0 .. n-1 of the chunk at `p`, in this or (reverse) the other order.  The buffer's bounds give zeros
    // past the width and (but for rows that overlap by their stride) for what lies behind the last row or, as
    // an unsigned offset, before the first.
    __device__ __forceinline__ void load(const char *p, int stride, int at, int n, int row_end, bool reverse) {
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(p), (short)0,
                                                            (n - 1) * stride + row_end, 0x00020000);
        uint32_t off = (uint32_t)at + (reverse ? (uint32_t)((n - 1) * stride) : 0u);
        const uint32_t step = (uint32_t)(reverse ? -rpp * stride : rpp * stride);
#pragma unroll
        for (int i = 0; i < passes; ++i) {
            r[i] = mx::buf_ld16(rsrc, (int)off);
            off += step;
        }
    }
    __device__ __forceinline__ void store(typename T::lds *s) const {
        const int pc = threadIdx.x % pieces, r0 = threadIdx.x / pieces;
#pragma unroll
        for (int i = 0; i < passes; ++i) {
            typename T::lds *row = s + (r0 + i * rpp) * ld;
            if constexpr (BF16 && ORD == kRows) {
                // channels 8 pc .. + 7 of the row: quads 2 q and 2 q + 1 of a 32-block (q = pc % 4), of which quad
                // j is the first (j < 4) or second half of lane group j % 4's fragment
                const int q = pc & 3;
                typename T::lds *at = s + (r0 + i * rpp) * prow + 8 * (pc >> 2) + 4 * (q >> 1);
                const int to = (2 * q) & 3;
                *reinterpret_cast<uint2 *>(at + to * plane + 32 * to) = make_uint2(r[i].x, r[i].y);
                *reinterpret_cast<uint2 *>(at + (to + 1) * plane + 32 * to) = make_uint2(r[i].z, r[i].w);
            } else {
                *reinterpret_cast<uint4 *>(row + pc * per) = r[i];
            }
        }
    }
};

__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 c) {
    return bf16x8{a[0], a[1], a[2], a[3], c[0], c[1], c[2], c[3]};
}
// Fragment of row `row`, channel block kb, of a tile of the type TILE.
template <bool BF16, Order ORD, typename TILE>
__device__ __forceinline__ typename El<BF16>::frag row_frag(const typename El<BF16>::lds *s, int row, int kb, int lg) {
    constexpr int ld = TILE::ld;
    if constexpr (!BF16) {
        return *reinterpret_cast<const f32x4 *>(s + row * ld + 16 * kb + 4 * lg);
    } else if constexpr (ORD == kRows) {
        return *reinterpret_cast<const bf16x8 *>(s + lg * TILE::plane + 64 * (lg >> 1) + row * TILE::prow + 8 * kb);
    } else {
        const __bf16 *at = s + row * ld + 32 * kb + 4 * lg;
        return join(*reinterpret_cast<const bf16x4 *>(at), *reinterpret_cast<const bf16x4 *>(at + 16));
    }
}
// Fragment over the tokens of block kb, of the 16 channels from col on (as they lie in LDS: lane lr has col + lr).
template <bool BF16>
__device__ __forceinline__ typename El<BF16>::frag col_frag(const typename El<BF16>::lds *s, int ld, int col, int kb,
                                                            int lr, int lg) {
    if constexpr (BF16) {
        const __bf16 *at = s + (32 * kb + 4 * lg + (lr >> 2)) * ld + col + 4 * (lr & 3);
        return join(mx::lds_read_tr(at), mx::lds_read_tr(at + 16 * ld));
    } else {
        f32x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = s[(16 * kb + 4 * lg + e) * ld + col + lr];
        return x;
    }
}

// Two fp32 values rounded to bf16, packed; as two terms (x = hi + lo to 2^-17) and what hi leaves.
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack2(float x0, float x1) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{x0, x1}), mx::bf16x2));
}
__device__ __forceinline__ void rest2(float &x0, float &x1, uint32_t hi) {
    x0 -= __uint_as_float(hi << 16);
    x1 -= __uint_as_float(hi & 0xffff0000u);
}
// Two stacked tiles of an accumulator as a fragment in two terms.
__device__ __forceinline__ void split_tiles(f32x4 t0, f32x4 t1, bf16x8 &hi, bf16x8 &lo) {
    float x[8] = {t0[0], t0[1], t0[2], t0[3], t1[0], t1[1], t1[2], t1[3]};
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        h[e] = pack2(x[2 * e], x[2 * e + 1]);
        rest2(x[2 * e], x[2 * e + 1], h[e]);
        l[e] = pack2(x[2 * e], x[2 * e + 1]);
    }
    hi = __builtin_bit_cast(bf16x8, make_uint4(h[0], h[1], h[2], h[3]));
    lo = __builtin_bit_cast(bf16x8, make_uint4(l[0], l[1], l[2], l[3]));
}
// Eight fp32 values as three bf16 terms, 24 bits: x = hi + mid + lo to fp32's own rounding.
__device__ __forceinline__ void split8x3(float *x, bf16x8 &hi, bf16x8 &mid, bf16x8 &lo) {
    uint32_t h[4], m[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        h[e] = pack2(x[2 * e], x[2 * e + 1]);
        rest2(x[2 * e], x[2 * e + 1], h[e]);
        m[e] = pack2(x[2 * e], x[2 * e + 1]);
        rest2(x[2 * e], x[2 * e + 1], m[e]);
        l[e] = pack2(x[2 * e], x[2 * e + 1]);
    }
    hi = __builtin_bit_cast(bf16x8, make_uint4(h[0], h[1], h[2], h[3]));
    mid = __builtin_bit_cast(bf16x8, make_uint4(m[0], m[1], m[2], m[3]));
    lo = __builtin_bit_cast(bf16x8, make_uint4(l[0], l[1], l[2], l[3]));
}

// The pair matrix's fragment of token tile I, token block kb (bf16: kb <= I / 2; fp32: kb <= I).
template <bool BF16, int CI>
__device__ __forceinline__ int pair_frag(int I, int kb) {
    if constexpr (BF16) return CI == 2 ? I : mx::lower_frag(I, kb);
    else return I * CI + kb;
}

enum { kSums = 0, kWalk = 1, kWalkDg = 2 };

template <bool BF16, int PAD, int CH, int WV, int MODE>
struct Smem {
    using L = typename El<BF16>::lds;
    static constexpr int nfrag = BF16 ? (CH == 64 ? 6 : 2) : (CH / 16) * (CH / 16);
    __align__(16) L a[MODE == kSums ? 1 : Tile<BF16, PAD, CH, kRows, WV>::size];
    __align__(16) L b[CH * Tile<BF16, PAD, CH, kBoth, WV>::ld];
    __align__(16) L c[CH * Tile<BF16, 16 * WV, CH, kColumns, WV>::ld];
    __align__(16) char p[MODE == kSums ? 16 : nfrag * 1024];
    __align__(16) char ph[MODE == kWalkDg ? nfrag * 1024 : 16];  // (i - j) times the pair matrix, hi
    __align__(16) char pl[MODE == kWalkDg ? nfrag * 1024 : 16];  // and lo
    __align__(16) float rpow[2 * CH + 8];                        // lambda^(CH - y), 0 behind
    __align__(16) float write[CH];                               // what token j's write is multiplied by
    double dg[WV];
    PlaceSmem place;
};

template <bool BF16, int PAD, int CH, int WV, int MODE>
__global__ __launch_bounds__(64 * WV, WV == 8 && MODE != kWalkDg ? 4 : 2) void walk_kernel(WalkSet set) {
    using T = El<BF16>;
    using frag = typename T::frag;
    constexpr int KD = PAD / T::depth;   // channel blocks of a row
    constexpr int KT = CH / T::depth;    // token blocks of a chunk
    constexpr int CI = CH / 16;          // token tiles of a chunk
    constexpr int TT = PAD / 16;         // row tiles of the state
    constexpr int COLS = 16 * WV;
    constexpr bool OUT = MODE != kSums, DG = MODE == kWalkDg;
    using TileA = Tile<BF16, PAD, CH, kRows, WV>;
    using TileB = Tile<BF16, PAD, CH, kBoth, WV>;
    using TileC = Tile<BF16, COLS, CH, kColumns, WV>;
    constexpr int LDB = TileB::ld, LDC = TileC::ld;
    __shared__ Smem<BF16, PAD, CH, WV, MODE> sm;

    const Walk &w = set.w[blockIdx.y];
    const Batch &b = set.b;
    const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lg = lane >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    int group, slice;
    mx::state_slot(blockIdx.x, b.units * b.H, set.slices, group, slice);
    const int u = group / b.H, h = group - u * b.H;
    const Place pl = find_place<CH, DG, WV>(b, u, sm.place);
    const size_t part = ((size_t)u * b.H + h) * set.slices + slice;  // of u, chunk_e, dg_part
    const int col0 = slice * COLS + wv * 16;                         // the wavefront's first column
    if (OUT && b.cu && w.zero_outside && u == 0) {
        const int es = w.out_f32 ? 4 : T::bytes, per = 16 / es;
        const int cols = min(COLS, w.Dc - slice * COLS);
        const int outside = pl.first + (b.T - pl.last);
        for (int64_t x = tid; x < (int64_t)outside * (cols / per); x += 64 * WV) {
            const int i = (int)(x / (cols / per)), row = i < pl.first ? i : pl.last + (i - pl.first);
            char *dst = w.out + (((int64_t)row * b.H + h) * w.Dc + slice * COLS + (x % (cols / per)) * per) * es;
            *reinterpret_cast<uint4 *>(dst) = make_uint4(0, 0, 0, 0);
        }
    }
    if (pl.n < 0 || slice * COLS >= w.Dc) {
        if (DG && w.dg_part && tid == 0) w.dg_part[part] = 0.0;
        return;
    }

    const bool last_seg = w.reverse ? pl.s == 0 : pl.s == pl.ns - 1;
    if (!OUT && last_seg) return;  // no segment starts from its sum

    const float g = b.g[h];
    for (int y = tid; y < 2 * CH + 8; y += 64 * WV) sm.rpow[y] = y <= CH ? decay_power(g, CH - y) : 0.f;
    auto lam = [&](int x) { return sm.rpow[CH - x]; };  // lambda^x, 0 <= x <= CH
    if constexpr (OUT && BF16) {
        // the upper tiles inside the fragments' 32-blocks stay zero
        for (int x = tid; x < Smem<BF16, PAD, CH, WV, MODE>::nfrag * 64; x += 64 * WV) {
            const int I = CI == 2 ? x / 64 : mx::frag_M(x / 64), kb = CI == 2 ? 0 : mx::frag_kb(x / 64);
            if (2 * kb + 1 > I) {
                *reinterpret_cast<uint4 *>(sm.p + x * 16) = make_uint4(0, 0, 0, 0);
                if constexpr (DG) {
                    *reinterpret_cast<uint4 *>(sm.ph + x * 16) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(sm.pl + x * 16) = make_uint4(0, 0, 0, 0);
                }
            }
        }
    }
    __syncthreads();

    // ---- the rows of the segment, and its first chunk's loads
    const int chunks = (pl.len + CH - 1) / CH;
    const char *pa = nullptr, *pb, *pc;
    const int64_t tok = pl.tok0 + pl.t0;
    auto view = [&](const View &v) { return v.p + (b.cu ? 0 : pl.n * v.seq) + (h / v.div) * v.head + tok * v.tok; };
    if constexpr (OUT) pa = view(w.a);
    pb = view(w.b);
    pc = view(w.c);
    const int sa = (int)w.a.tok, sb = (int)w.b.tok, sc = (int)w.c.tok;
    // (row strides of a chunk fit 32 bits; a reversed chunk's rows lie at n-1-r)
    const int rsgn = w.reverse ? -1 : 1;
    const int fa = TileA::first(rsgn * sa, 0, w.Da), fb = TileB::first(rsgn * sb, 0, w.Da);
    const int fc = TileC::first(rsgn * sc, slice * COLS, w.Dc);
    TileA ta;
    TileB tb;
    TileC tc;
    auto fetch = [&](int x) {
        const int ci = w.reverse ? chunks - 1 - x : x;
        const int n = min(CH, pl.len - ci * CH);
        const int64_t row = ci * CH;
        if constexpr (OUT) ta.load(pa + row * w.a.tok, sa, fa, n, w.Da * T::bytes, w.reverse);
        tb.load(pb + row * w.b.tok, sb, fb, n, w.Da * T::bytes, w.reverse);
        tc.load(pc + row * w.c.tok, sc, fc, n, w.Dc * T::bytes, w.reverse);
    };
    // (beside the state only where the registers hold both)
    constexpr bool early = !(BF16 && PAD == 128 && WV == 8 && MODE == kWalk);
    if (early && chunks > 0) fetch(0);

    // ---- the entering state
        const size_t e_base = ((size_t)pl.n * b.H + h) * w.Da * w.Dc;
    f32x4 E[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t)
        E[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto fragments = [&](float *base, size_t index, int t) {
        return reinterpret_cast<f32x4 *>(base + index * (size_t)(PAD * COLS)) + (wv * TT + t) * 64 + lane;
    };
    if constexpr (OUT) {
        if (w.e0) {
            const float f = w.e0_decay ? lam(1) : 1.f;
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int row = 16 * t + 4 * lg, col = col0 + lr;
                if (row < w.Da && col < w.Dc) {
                    if (w.e0_t) {
                        E[t] = *reinterpret_cast<const f32x4 *>(w.e0 + e_base + (size_t)col * w.Da + row);
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r) E[t][r] = w.e0[e_base + (size_t)(row + r) * w.Dc + col];
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) E[t][r] *= f;
                }
            }
        }
    }
    if constexpr (OUT) {
        // the segments before this one, two of them in flight
        const int before = w.reverse ? pl.ns - 1 - pl.s : pl.s;
        auto number = [&](int x) { return w.reverse ? pl.ns - 1 - x : x; };
        auto load_sum = [&](int x, f32x4 (&to)[TT]) {
            const size_t index = ((size_t)(u - pl.s + number(x)) * b.H + h) * set.slices + slice;
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                // (a transposed sum holds the state's own rows and columns only)
                to[t] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (16 * t + 4 * lg < w.Da && col0 + lr < w.Dc) to[t] = *fragments(w.u, index, t);
            }
        };
        auto add_sum = [&](int x, const f32x4 (&from)[TT]) {
            const float f = decay_power(g, min(b.seg, pl.seq_len - number(x) * b.seg));
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) E[t][r] = f * E[t][r] + from[t][r];
        };
        for (int x = 0; x < before; x += 2) {
            f32x4 U0[TT], U1[TT];
            load_sum(x, U0);
            if (x + 1 < before) load_sum(x + 1, U1);
            add_sum(x, U0);
            if (x + 1 < before) add_sum(x + 1, U1);
        }
    }

    // ---- the walk
    // The wavefront's pair tiles, PT side by side: four wavefronts have three of ten (one with two takes its first
    // again), eight have one and then the two last ones, and of three tiles each has one.
    constexpr int PT = CI == 4 && WV == 4 ? 3 : 1;
    const int pair_rounds = CI == 4 ? (WV == 8 && wv < 2 ? 2 : 1) : wv < 3 ? 1 : 0;
    int tile_i[PT], tile_j[PT];
    if constexpr (PT == 3) {
        tile_i[0] = wv < 2 ? 3 : 2, tile_j[0] = 2 * (wv & 1);                            // 3,0 3,2 2,0 2,2
        tile_i[1] = wv < 2 ? 3 : 4 - wv, tile_j[1] = wv == 0 ? 1 : wv == 1 ? 3 : 3 - wv;  // 3,1 3,3 2,1 1,0
        tile_i[2] = wv < 2 ? wv : 2, tile_j[2] = wv < 2 ? wv : 2 * (wv & 1);              // 0,0 1,1 again
    }
    // lambda^(i-j) of a lane's elements of a tile on the diagonal and of the one before it, with the scale; the
    // tiles farther apart by a factor (all powers >= 0: none overflows)
    f32x4 near0, near1;
    {
        const float pscale = w.oscale * w.uscale;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int d = lr - 4 * lg - r;
            near0[r] = lam(max(d, 0)) * pscale;
            near1[r] = lam(16 + d) * pscale;
        }
    }
    const float lam16 = CI > 2 ? lam(16) : 1.f, lam32 = CI > 2 ? lam(32) : 1.f;
    const int oes = w.out_f32 ? 4 : T::bytes;
    const int fo = col0 + 4 * lg < w.Dc ? rsgn * lr * (b.H * w.Dc * oes) + (col0 + 4 * lg) * oes : kFar;
    const bool weighted = DG && w.x.p && !w.reverse;  // the walk that sums (i - j) times the pairs
    double dg = 0.0;
    if (!early && chunks > 0) fetch(0);
    for (int x = 0; x < chunks; ++x) {
        const int ci = w.reverse ? chunks - 1 - x : x;
        const int n = min(CH, pl.len - ci * CH);
        // (barriers of the loop wait for LDS only: the next chunk's loads and this one's stores stay in flight)
        mx::barrier_lds();  // the tiles of the chunk before are read
        if constexpr (OUT) ta.store(sm.a);
        tb.store(sm.b);
        tc.store(sm.c);
        const bool end = last_seg && x + 1 == chunks;       // nothing reads E after it but the caller
        const int less = end && !w.reverse && OUT ? 1 : 0;  // S, not lambda S
        const bool update = !OUT || !end || w.ef;
        // token j's write still decays n - less - j times
        if ((x < 2 || n < CH || less) && tid < CH) sm.write[tid] = tid < n ? sm.rpow[CH - n + less + tid] * w.uscale : 0.f;
        if (x + 1 < chunks) fetch(x + 1);
        mx::barrier_lds();
        // the state that dq's walk kept of this chunk, on the way while the pairs and the state's read are formed
        const size_t kept_at = ((size_t)(pl.chunk0 + ci) * b.H + h) * set.slices + slice;
        f32x4 kept[DG ? TT : 1];
        if constexpr (DG) {
            if (w.chunk_e && w.reverse) {
#pragma unroll
                for (int t = 0; t < TT; ++t)
                    kept[t] = *fragments(w.chunk_e, kept_at, t);
            }
        }
        // and the lane's part of the rows of x: four channels of each token
        f32x4 xr[DG ? CI : 1];
        if constexpr (DG) {
            if (w.x.p) {
                const char *px = view(w.x);
#pragma unroll
                for (int I = 0; I < CI; ++I) {
                    const int i = 16 * I + lr, col = col0 + 4 * lg;
                    xr[I] = f32x4{0.f, 0.f, 0.f, 0.f};
                    if (i < n && col < w.Dc) {
                        const int64_t row = ci * CH + (w.reverse ? n - 1 - i : i);
                        const char *at = px + row * w.x.tok + (int64_t)col * T::bytes;
                        if constexpr (BF16) {
                            const uint2 y = *reinterpret_cast<const uint2 *>(at);
                            xr[I] = f32x4{__uint_as_float(y.x << 16), __uint_as_float(y.x & 0xffff0000u),
                                              __uint_as_float(y.y << 16), __uint_as_float(y.y & 0xffff0000u)};
                        } else {
                            xr[I] = *reinterpret_cast<const f32x4 *>(at);
                        }
                    }
                }
            }
        }

        if constexpr (OUT) {
            // pair tiles (I, J), J <= I, transposed (rows: tokens j, columns: tokens i)
            for (int round = 0; round < pair_rounds; ++round) {
                if constexpr (PT == 1) {
                    const int t = wv + 8 * round;
                    tile_i[0] = t >= 6 ? 3 : t >= 3 ? 2 : t >= 1 ? 1 : 0;
                    tile_j[0] = t - tile_i[0] * (tile_i[0] + 1) / 2;
                }
            f32x4 acc[PT];
#pragma unroll
            for (int q = 0; q < PT; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < KD; ++kb)
#pragma unroll
                for (int q = 0; q < PT; ++q)
                    acc[q] = mul_add(row_frag<BF16, kBoth, TileB>(sm.b, 16 * tile_j[q] + lr, kb, lg),
                                     row_frag<BF16, kRows, TileA>(sm.a, 16 * tile_i[q] + lr, kb, lg), acc[q]);
#pragma unroll
            for (int q = 0; q < PT; ++q) {
                const int I = tile_i[q], J = tile_j[q], apart = I - J;
                f32x4 val, wgt;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float f = apart == 0 ? near0[r] : near1[r] * (apart == 1 ? 1.f : apart == 2 ? lam16 : lam32);
                    val[r] = apart > 0 || lr >= 4 * lg + r ? acc[q][r] * f : 0.f;
                    wgt[r] = val[r] * static_cast<float>(16 * apart + lr - 4 * lg - r);
                }
                if constexpr (BF16) {
                    const int at = (pair_frag<BF16, CI>(I, J >> 1) * 64 + lane) * 16 + (J & 1) * 8;
                    *reinterpret_cast<uint2 *>(sm.p + at) = make_uint2(pack2(val[0], val[1]), pack2(val[2], val[3]));
                    if (DG && weighted) {
                        uint2 hi, lo;
                        mx::split2(wgt[0], wgt[1], hi.x, lo.x);
                        mx::split2(wgt[2], wgt[3], hi.y, lo.y);
                        *reinterpret_cast<uint2 *>(sm.ph + at) = hi;
                        *reinterpret_cast<uint2 *>(sm.pl + at) = lo;
                    }
                } else {
                    const int at = (pair_frag<BF16, CI>(I, J) * 64 + lane) * 16;
                    *reinterpret_cast<f32x4 *>(sm.p + at) = val;
                    if (DG && weighted) *reinterpret_cast<f32x4 *>(sm.ph + at) = wgt;
                }
            }
            }
        }

        f32x4 O[CI];
        if constexpr (OUT) {
            // the state's read, transposed: rows c's channels, columns tokens.  From here to the barrier a
            // wavefront is mostly products: it goes first (the prefill walk's passes 122 -> 118 us)
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int I = 0; I < CI; ++I)
                O[I] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < KD; ++kb) {
                frag hi, lo;
                if constexpr (BF16) split_tiles(E[2 * kb], E[2 * kb + 1], hi, lo);
                else hi = E[kb];
#pragma unroll
                for (int I = 0; I < CI; ++I) {
                    const frag af = row_frag<BF16, kRows, TileA>(sm.a, 16 * I + lr, kb, lg);
                    O[I] = mul_add(hi, af, O[I]);
                    if constexpr (BF16) O[I] = mul_add(lo, af, O[I]);
                }
            }
#pragma unroll
            for (int I = 0; I < CI; ++I) {
                const float f = lam(16 * I + lr) * w.oscale;
#pragma unroll
                for (int r = 0; r < 4; ++r) O[I][r] *= f;
            }
        }

        if constexpr (DG) {
            if (w.chunk_e) {
                float sum = 0.f;
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    if (!w.reverse) {
                        *fragments(w.chunk_e, kept_at, t) = E[t];
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r) sum += kept[t][r] * E[t][r];
                    }
                }
                // pairs across the whole chunk: n lambda^n <S, R>, and the stored E is lambda S
                if (w.reverse) dg += static_cast<double>(sum) * static_cast<double>(n * lam(n - 1));
            }
        }
        if (update) {
            const float f = lam(n - less);
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) E[t][r] *= f;
        }
        f32x4 Y[DG ? CI : 1];
        if constexpr (DG)
#pragma unroll
            for (int I = 0; I < CI; ++I)
                Y[I] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (DG) {
            // the state's part of <x, out>, token i weighted by its distance to the chunk's start (in the
            // direction that the pairs decay)
            if (w.x.p) {
                float sum = 0.f;
#pragma unroll
                for (int I = 0; I < CI; ++I) {
                    const int i = 16 * I + lr;
                    const float f = static_cast<float>(w.reverse ? i : i + 1);
                    if (i < n) {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (col0 + 4 * lg < w.Dc) sum += f * xr[I][r] * O[I][r];
                    }
                }
                dg += static_cast<double>(sum);
            }
        }
        // (c is read twice, here and behind the barrier: kept, it would not fit the registers)
        auto c_frags = [&](int kb, frag &to) {
            to = col_frag<BF16>(sm.c, LDC, wv * 16, kb, lr, lg);
        };
        if (update) {
#pragma unroll
            for (int kb = 0; kb < KT; ++kb) {
                frag cf, wh, wm, wl;
                c_frags(kb, cf);
                f32x4 wj[T::depth / 16];
#pragma unroll
                for (int y = 0; y < T::depth / 16; ++y)
                    wj[y] = *reinterpret_cast<const f32x4 *>(sm.write + T::depth * kb + 16 * y + 4 * lg);
                if constexpr (BF16) {
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = static_cast<float>(cf[e]) * wj[e / 4][e % 4];
                    split8x3(y, wh, wm, wl);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) wh[e] = cf[e] * wj[0][e];
                }
                frag bt = col_frag<BF16>(sm.b, LDB, 0, kb, lr, lg);
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const frag now = bt;
                    if (t + 1 < TT) bt = col_frag<BF16>(sm.b, LDB, 16 * (t + 1), kb, lr, lg);
                    E[t] = mul_add(now, wh, E[t]);
                    if constexpr (BF16) {
                        E[t] = mul_add(now, wm, E[t]);
                        E[t] = mul_add(now, wl, E[t]);
                    }
                }
            }
        }

        if constexpr (OUT) {
            __builtin_amdgcn_s_setprio(0);
            mx::barrier_lds();  // the pair matrix is written
#pragma unroll
            for (int kb = 0; kb < KT; ++kb) {
                frag cf;
                c_frags(kb, cf);
#pragma unroll
                for (int I = 0; I < CI; ++I) {
                    if (BF16 ? kb <= (I >> 1) : kb <= I) {
                        const int at = (pair_frag<BF16, CI>(I, kb) * 64 + lane) * 16;
                        const frag pf = *reinterpret_cast<const frag *>(sm.p + at);
                        O[I] = mul_add(cf, pf, O[I]);
                        if constexpr (DG) {
                            if (weighted) {
                                const frag qh = *reinterpret_cast<const frag *>(sm.ph + at);
                                Y[I] = mul_add(cf, qh, Y[I]);
                                if constexpr (BF16) {
                                    const frag ql = *reinterpret_cast<const frag *>(sm.pl + at);
                                    Y[I] = mul_add(cf, ql, Y[I]);
                                }
                            }
                        }
                    }
                }
            }
            // rows of the chunk: offsets as in Tile::load, stores past the bounds are dropped
            const int64_t row0 = (int64_t)(b.cu ? 0 : (int64_t)pl.n * b.T) + tok + ci * CH;
            const int orow = b.H * w.Dc * oes;
            const auto ro = __builtin_amdgcn_make_buffer_rsrc(w.out + (row0 * b.H + h) * w.Dc * oes, (short)0,
                                                              (n - 1) * orow + w.Dc * oes, 0x00020000);
#pragma unroll
            for (int I = 0; I < CI; ++I) {
                const uint32_t off = w.reverse ? (uint32_t)fo + (uint32_t)((n - 1 - 16 * I) * orow)
                                               : (uint32_t)fo + (uint32_t)(16 * I * orow);
                typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
                typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
                if (!BF16 || w.out_f32) {
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[I]), ro, (int)off, 0, 0);
                } else {
                    const u32x2 v = {pack2(O[I][0], O[I][1]), pack2(O[I][2], O[I][3])};
                    __builtin_amdgcn_raw_buffer_store_b64(v, ro, (int)off, 0, 0);
                }
                if constexpr (DG) {
                    if (weighted && 16 * I + lr < n) {
                        float sum = 0.f;
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (col0 + 4 * lg < w.Dc) sum += xr[I][r] * Y[I][r];
                        dg += static_cast<double>(sum);
                    }
                }
            }
        }
    }

    if constexpr (!OUT) {
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            *fragments(w.u, part, t) = E[t];
            if (w.u_t) {
                // element (row, col) as (col, row) of the other walk's fragments
                const int row = 16 * t + 4 * lg, col = col0 + lr;
                const int ws = row / COLS, ww = row % COLS / 16, cc = row % 16;
                float *to = w.u_t + (((size_t)u * b.H + h) * set.slices + ws) * (size_t)(PAD * COLS) +
                            (((size_t)ww * TT + (col >> 4)) * 64 + (col >> 2 & 3) * 16 + cc) * 4 + (col & 3);
                if (row < w.Da && col < w.Dc) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) to[4 * r] = E[t][r];
                }
            }
        }
    } else {
        if (w.ef && last_seg) {
            // an empty sequence keeps its state: E holds e0, decayed in the forward direction
            const bool empty = pl.seq_len == 0;
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int row = 16 * t + 4 * lg, col = col0 + lr;
                if (row < w.Da && col < w.Dc) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const size_t at = e_base + (size_t)(row + r) * w.Dc + col;
                        w.ef[at] = empty ? (w.e0 ? w.e0[at] : 0.f) : E[t][r];
                    }
                }
            }
        }
        if constexpr (DG) {
            if (w.dg_part) {
#pragma unroll
                for (int off = 32; off > 0; off >>= 1) dg += __shfl_xor(dg, off, 64);
                if (lane == 0) sm.dg[wv] = dg;
                __syncthreads();
                if (tid == 0)
                    {
                    double all = 0.0;
                    for (int i = 0; i < WV; ++i) all += sm.dg[i];
                    w.dg_part[part] = all;
                }
            }
        }
    }
}

template <bool BF16, int PAD, int CH, int WV, int MODE>
hipError_t launch(const WalkSet &s, hipStream_t stream) {
    const dim3 grid((unsigned)(s.b.units * s.b.H * s.slices), (unsigned)s.count);
    hipLaunchKernelGGL((walk_kernel<BF16, PAD, CH, WV, MODE>), grid, dim3(64 * WV), 0, stream, s);
    return hipGetLastError();
}

template <int MODE>
hipError_t dispatch(const WalkSet &s, bool bf16, const Shape &sh, hipStream_t stream) {
    if (bf16) {
        if (sh.pad == 64)
            return sh.cols == 64 ? launch<true, 64, 64, 4, MODE>(s, stream) : launch<true, 64, 64, 8, MODE>(s, stream);
        if (sh.pad == 128)
            return sh.cols == 64 ? launch<true, 128, 64, 4, MODE>(s, stream) : launch<true, 128, 64, 8, MODE>(s, stream);
        return launch<true, 256, 32, 4, MODE>(s, stream);
    }
    if (sh.pad == 64)
        return sh.cols == 64 ? launch<false, 64, 32, 4, MODE>(s, stream) : launch<false, 64, 32, 8, MODE>(s, stream);
    if (sh.pad == 128)
        return sh.cols == 64 ? launch<false, 128, 32, 4, MODE>(s, stream) : launch<false, 128, 32, 8, MODE>(s, stream);
    return launch<false, 256, 32, 4, MODE>(s, stream);
}

// ---- sums over the query heads of a group, and of dL/dg's parts
template <bool BF16>
__global__ __launch_bounds__(kThreads) void group_sum_kernel(GroupSum k, GroupSum v, int G) {
    const GroupSum &s = blockIdx.y == 0 ? k : v;
    const size_t x = (size_t)blockIdx.x * kThreads + threadIdx.x;
    if (x >= s.rows * (s.width / 4)) return;
    const size_t row = x / (s.width / 4), col = x % (s.width / 4) * 4;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < G; ++i) {
        const float4 y = *reinterpret_cast<const float4 *>(s.src + (row * G + i) * s.width + col);
        sum.x += y.x; sum.y += y.y; sum.z += y.z; sum.w += y.w;
    }
    const size_t at = row * s.width + col;
    store_out<BF16>(s.dst, at, sum.x);
    store_out<BF16>(s.dst, at + 1, sum.y);
    store_out<BF16>(s.dst, at + 2, sum.z);
    store_out<BF16>(s.dst, at + 3, sum.w);
}

__global__ __launch_bounds__(kThreads) void dg_sum_kernel(const double *__restrict__ part, float *__restrict__ dg,
                                                          int units, int H, int slices, int walks, size_t stride) {
    __shared__ double red[kThreads];
    const int h = blockIdx.x;
    double sum = 0.0;
    for (int w = 0; w < walks; ++w)
        for (size_t x = threadIdx.x; x < (size_t)units * slices; x += kThreads)
            sum += part[w * stride + ((x / slices) * H + h) * slices + x % slices];
    red[threadIdx.x] = sum;
    __syncthreads();
    for (int off = kThreads / 2; off > 0; off >>= 1) {
        if ((int)threadIdx.x < off) red[threadIdx.x] += red[threadIdx.x + off];
        __syncthreads();
    }
    if (threadIdx.x == 0) dg[h] = static_cast<float>(red[0]);
}

}  // namespace

Shape shape_of(bool bf16, int wide, int cols) {
    const int chunk = bf16 && wide <= 128 ? 64 : 32;
    if (wide > 128) return Shape{256, chunk, 64, 2};
    const bool both = cols > 64;  // eight wavefronts
    return Shape{wide <= 64 ? 64 : 128, chunk, both ? 128 : 64, 2};
}
size_t frag_bytes(const Shape &s, int slices) { return (size_t)s.pad * s.cols * slices * sizeof(float); }

hipError_t launch_segment_sums(const WalkSet &s, bool bf16, const Shape &sh, hipStream_t stream) {
    return dispatch<kSums>(s, bf16, sh, stream);
}
hipError_t launch_walks(const WalkSet &s, bool bf16, const Shape &sh, bool dg, hipStream_t stream) {
    return dg ? dispatch<kWalkDg>(s, bf16, sh, stream) : dispatch<kWalk>(s, bf16, sh, stream);
}
hipError_t launch_group_sums(const GroupSum &k, const GroupSum &v, bool bf16, int G, hipStream_t stream) {
    const size_t quads = k.rows * (std::max(k.width, v.width) / 4);
    if (quads == 0) return hipSuccess;
    const dim3 grid((unsigned)((quads + kThreads - 1) / kThreads), 2);
    if (bf16) hipLaunchKernelGGL(group_sum_kernel<true>, grid, dim3(kThreads), 0, stream, k, v, G);
    else hipLaunchKernelGGL(group_sum_kernel<false>, grid, dim3(kThreads), 0, stream, k, v, G);
    return hipGetLastError();
}
hipError_t launch_dg_sum(const double *part, float *dg, int units, int H, int slices, int walks, size_t stride,
                         hipStream_t stream) {
    hipLaunchKernelGGL(dg_sum_kernel, dim3((unsigned)H), dim3(kThreads), 0, stream, part, dg, units, H, slices, walks,
                       stride);
    return hipGetLastError();
}

}  // namespace hd
}  // namespace gdr
