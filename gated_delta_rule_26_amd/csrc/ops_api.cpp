// C ABI of the per-head-decay and beam-search operators: argument validation (host code, before any HIP
// call), the plan of a call (tiles, segments, workspace) and its launches.  See include/gdr_ops.h.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ops_internal.h"

namespace {

using gdr::hd::Batch;
using gdr::hd::Shape;
using gdr::hd::View;
using gdr::hd::Walk;
using gdr::hd::WalkSet;

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }
Range range_of(const void *p, size_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, p ? lo + bytes : lo};
}
bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <int NI, int NO>
bool alias_free(const Range (&in)[NI], const Range (&out)[NO]) {
    for (int i = 0; i < NO; ++i) {
        for (const Range &r : in)
            if (overlap(r, out[i])) return false;
        for (int j = 0; j < i; ++j)
            if (overlap(out[j], out[i])) return false;
    }
    return true;
}

constexpr int kFill = 256;  // compute units

constexpr size_t kMost = (size_t)1 << 46;  // elements of a tensor, and of a stride

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

int check_desc(const gdr_head_decay_desc *d, bool step) {
    if (!d) return GDR_E_NULL;
    if (d->dtype != GDR_F32 && d->dtype != GDR_BF16) return GDR_E_MODE;
    if (!std::isfinite(d->scale)) return GDR_E_MODE;
    if (d->B < 0 || d->H < 0 || d->Hk < 0 || (!step && d->T < 0)) return GDR_E_SHAPE;
    if (d->H > 0 && (d->Hk == 0 || d->H % d->Hk != 0)) return GDR_E_SHAPE;
    if (d->Dk < 8 || d->Dk > gdr::hd::kMaxWidth || d->Dk % 8 || d->Dv < 8 || d->Dv > gdr::hd::kMaxWidth || d->Dv % 8)
        return GDR_E_UNSUPPORTED;
    // the outputs' rows of a chunk are addressed with 32-bit byte offsets
    if (d->H > 16384) return GDR_E_SHAPE;
    const double tokens = (step ? 1.0 : (double)d->T) * (d->B > 0 ? d->B : 1);
    if (tokens * d->H * 256.0 > (double)kMost || (double)d->B * d->H * 65536.0 > (double)kMost) return GDR_E_SHAPE;
    return GDR_OK;
}

// A strided input [B or 1, T, heads, width]: bounds and alignment of the strides; its byte range.
int check_view(const void *p, const int64_t *stride, int B, int T, int heads, int width, int es, Range *r, View *v,
               int div) {
    if (!p) return GDR_E_NULL;
    if (!aligned(p, 16)) return GDR_E_ALIGN;
    const int size[3] = {B, T, heads};
    // the rows of a chunk (64 tokens) are addressed with 32-bit byte offsets
    if (T > 1 && stride[1] > (int64_t)(1 << 24) / es) return GDR_E_SHAPE;
    int64_t far = width, step[3];
    for (int i = 0; i < 3; ++i) {
        step[i] = size[i] > 1 ? stride[i] : 0;  // a stride that is not taken does not matter
        if (step[i] < 0 || step[i] > (int64_t)kMost) return GDR_E_SHAPE;
        if (step[i] * es % 16) return GDR_E_ALIGN;
        const double reach = (double)far + (double)step[i] * (size[i] - 1);
        if (reach > (double)kMost) return GDR_E_SHAPE;
        if (size[i] > 0) far += step[i] * (size[i] - 1);
    }
    *r = range_of(p, (B > 0 && T > 0 && heads > 0) ? (size_t)far * es : 0);
    v->p = static_cast<const char *>(p);
    v->seq = step[0] * es;
    v->tok = step[1] * es;
    v->head = step[2] * es;
    v->div = div;
    return GDR_OK;
}

// How a call is cut up.  A workgroup walks a segment of a head and a column slice.  A segment costs a second
// reading of b and c and its sum, and all of them pay for a round of workgroups that is not full: so there are as
// many segments as fill the card once (what is resident at a time), of 64 tokens at least, and kMaxSegments per
// sequence at most (each starts from a chain of sums).  Measured: 1.5 times as many workgroups as the card holds
// 118 -> 130 us (prefill of 4 x 4096 tokens, 16 heads of 128 x 128), 5 segments instead of 6 for the backward pass
// of 2 x 8192 tokens (480 instead of 576 workgroups) 325 -> 273 us; segments of 64 instead of 256 tokens at least
// 171 -> 78 us (backward pass of 2 x 777 tokens, 4 heads, with dL/dg; 77 us now).
struct Plan {
    Shape sh;
    int slices;
    Batch b;
    bool sums;
    long chunks;  // of all sequences, at most
};

int make_plan(const gdr_head_decay_desc *d, bool packed, int wide, int cols, int walks, Plan *p) {
    p->sh = gdr::hd::shape_of(d->dtype == GDR_BF16, wide, cols);
    p->slices = (cols + p->sh.cols - 1) / p->sh.cols;
    const int64_t T = d->T;
    const int64_t share = (int64_t)kFill * p->sh.resident / std::max<int64_t>((int64_t)d->H * p->slices * walks, 1);
    int64_t seg, per = 1;
    if (packed) {
        // a sequence's last segment is half full on average; with many sequences the long ones among them are
        // still cut
        seg = T / std::max<int64_t>(std::max<int64_t>(share - d->B / 2, share / 2), 1);
        seg = std::max(seg, (T + gdr::hd::kMaxSegments - 1) / gdr::hd::kMaxSegments);
    } else {
        per = std::min<int64_t>(std::max<int64_t>(share / std::max(d->B, 1), 1), gdr::hd::kMaxSegments);
        seg = (T + per - 1) / per;
    }
    seg = std::max<int64_t>((seg + 63) / 64 * 64, 64);
    per = T > 0 ? (T + seg - 1) / seg : 1;
    const int64_t units = packed ? T / seg + d->B : per * d->B;
    // one workgroup per (unit, head, slice): the grid must stay below 2^31
    if ((double)units * d->H * p->slices >= 2147483648.0) return GDR_E_SHAPE;
    p->b = Batch();
    p->b.N = d->B;
    p->b.T = d->T;
    p->b.H = d->H;
    p->b.seg = (int)seg;
    p->b.units = (int)units;
    p->b.per_seq = packed ? 0 : (int)per;
    p->sums = packed ? T > seg : per > 1;
    p->chunks = packed ? T / p->sh.chunk + d->B : (T + p->sh.chunk - 1) / p->sh.chunk * d->B;
    return GDR_OK;
}

size_t state_count(const gdr_head_decay_desc *d) { return (size_t)d->B * d->H * d->Dk * d->Dv; }
size_t sum_bytes(const Plan &p) {
    return p.sums ? align256((size_t)p.b.units * p.b.H * gdr::hd::frag_bytes(p.sh, p.slices)) : 0;
}

int plan_fwd(const gdr_head_decay_desc *d, bool packed, Plan *p, size_t *bytes) {
    const int rc = make_plan(d, packed, d->Dk, d->Dv, 1, p);
    if (rc != GDR_OK) return rc;
    // with segments, an s0 that is also s_final is read from a copy: its segments start at their own times
    *bytes = p->sums ? sum_bytes(*p) + align256(state_count(d) * 4) : 0;
    return GDR_OK;
}

// Workspace of the backward pass, as offsets.
struct BwdSpace {
    size_t sums, part_k, part_v, chunk_e, dg, end;
};
int plan_bwd(const gdr_head_decay_desc *d, bool packed, bool need_dg, Plan *p, BwdSpace *s) {
    const int wide = d->Dk > d->Dv ? d->Dk : d->Dv;
    const int rc = make_plan(d, packed, wide, wide, need_dg ? 2 : 3, p);
    if (rc != GDR_OK) return rc;
    const size_t tokens = packed ? (size_t)d->T : (size_t)d->T * d->B;
    const bool shared = d->H != d->Hk;
    size_t at = 0;
    s->sums = at;
    at += 3 * sum_bytes(*p);
    s->part_k = at;
    at += shared ? align256(tokens * d->H * d->Dk * 4) : 0;
    s->part_v = at;
    at += shared ? align256(tokens * d->H * d->Dv * 4) : 0;
    s->chunk_e = at;
    at += need_dg ? align256((size_t)p->chunks * d->H * gdr::hd::frag_bytes(p->sh, p->slices)) : 0;
    s->dg = at;
    at += need_dg ? align256((size_t)p->b.units * d->H * p->slices * 2 * sizeof(double)) : 0;
    s->end = at;
    return GDR_OK;
}

int hip_status(hipError_t rc) { return rc == hipSuccess ? GDR_OK : GDR_E_HIP; }

}  // namespace

extern "C" {

int gdr_head_decay_fwd_workspace_size(const gdr_head_decay_desc *desc, int packed, size_t *bytes) {
    if (!bytes) return GDR_E_NULL;
    const int rc = check_desc(desc, false);
    if (rc != GDR_OK) return rc;
    Plan p;
    return plan_fwd(desc, packed != 0, &p, bytes);
}

int gdr_head_decay_fwd(const gdr_head_decay_desc *d, const int32_t *cu, const void *q, const void *k, const void *v,
                       const float *g, const float *s0, void *o, float *s_final, void *workspace,
                       size_t workspace_bytes, void *stream) {
    int rc = check_desc(d, false);
    if (rc != GDR_OK) return rc;
    const bool packed = cu != nullptr, bf16 = d->dtype == GDR_BF16;
    Plan p;
    size_t need = 0;
    rc = plan_fwd(d, packed, &p, &need);
    if (rc != GDR_OK) return rc;
    if (d->B == 0 || d->H == 0) return GDR_OK;
    const int es = bf16 ? 2 : 4, G = d->H / d->Hk, rows = packed ? 1 : d->B;
    Walk w;
    Range in[6] = {}, out[3] = {};
    if (d->T > 0) {
        if ((rc = check_view(q, d->q_stride, rows, d->T, d->H, d->Dk, es, &in[0], &w.a, 1)) != GDR_OK) return rc;
        if ((rc = check_view(k, d->k_stride, rows, d->T, d->Hk, d->Dk, es, &in[1], &w.b, G)) != GDR_OK) return rc;
        if ((rc = check_view(v, d->v_stride, rows, d->T, d->Hk, d->Dv, es, &in[2], &w.c, G)) != GDR_OK) return rc;
        if (!o) return GDR_E_NULL;
        if (need > 0 && (!workspace || workspace_bytes < need)) return GDR_E_WORKSPACE;
    }
    if (!g) return GDR_E_NULL;
    if (!aligned(g, 4) || !aligned(cu, 4) || !aligned(o, 16) || !aligned(s0, 16) || !aligned(s_final, 16) ||
        !aligned(workspace, 16))
        return GDR_E_ALIGN;
    const size_t state = state_count(d) * 4;
    in[3] = range_of(g, (size_t)d->H * 4);
    in[4] = range_of(cu, ((size_t)d->B + 1) * 4);
    in[5] = s0 == s_final ? range_of(nullptr, 0) : range_of(s0, state);
    out[0] = range_of(o, (size_t)rows * d->T * d->H * d->Dv * es);
    out[1] = range_of(s_final, state);
    out[2] = range_of(workspace, d->T > 0 ? need : 0);
    if (!alias_free(in, out)) return GDR_E_ALIAS;
    if (d->T == 0 && !s_final) return GDR_OK;

    const hipStream_t st = static_cast<hipStream_t>(stream);
    w.Da = d->Dk;
    w.Dc = d->Dv;
    w.oscale = d->scale;
    w.out = static_cast<char *>(o);
    w.e0 = s0;
    w.e0_decay = 1;
    w.ef = s_final;
    WalkSet set;
    set.b = p.b;
    set.b.cu = cu;
    set.b.g = g;
    set.count = 1;
    set.slices = p.slices;
    if (p.sums) {
        w.u = static_cast<float *>(workspace);
        if (s0 && s0 == s_final) {
            float *copy = reinterpret_cast<float *>(static_cast<char *>(workspace) + sum_bytes(p));
            if ((rc = hip_status(gdr::launch_state_init(copy, s0, state_count(d), st))) != GDR_OK) return rc;
            w.e0 = copy;
        }
    }
    set.w[0] = w;
    if (p.sums && (rc = hip_status(gdr::hd::launch_segment_sums(set, bf16, p.sh, st))) != GDR_OK) return rc;
    return hip_status(gdr::hd::launch_walks(set, bf16, p.sh, false, st));
}

int gdr_head_decay_bwd_workspace_size(const gdr_head_decay_desc *desc, int packed, int need_dg, size_t *bytes) {
    if (!bytes) return GDR_E_NULL;
    const int rc = check_desc(desc, false);
    if (rc != GDR_OK) return rc;
    Plan p;
    BwdSpace s;
    const int r2 = plan_bwd(desc, packed != 0, need_dg != 0, &p, &s);
    if (r2 == GDR_OK) *bytes = s.end;
    return r2;
}

int gdr_head_decay_bwd(const gdr_head_decay_desc *d, const int32_t *cu, const void *q, const void *k, const void *v,
                       const float *g, const float *s0, const void *d_o, const float *ds_final, void *dq, void *dk,
                       void *dv, float *dg, float *ds0, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_desc(d, false);
    if (rc != GDR_OK) return rc;
    const bool packed = cu != nullptr, bf16 = d->dtype == GDR_BF16, shared = d->H != d->Hk;
    Plan p;
    BwdSpace s;
    rc = plan_bwd(d, packed, dg != nullptr, &p, &s);
    if (rc != GDR_OK) return rc;
    if (d->B == 0 || d->H == 0) return GDR_OK;
    const int es = bf16 ? 2 : 4, G = d->H / d->Hk, rows = packed ? 1 : d->B;
    View vq, vk, vv, vo;
    Range in[8] = {}, out[6] = {};
    if (d->T > 0) {
        if ((rc = check_view(q, d->q_stride, rows, d->T, d->H, d->Dk, es, &in[0], &vq, 1)) != GDR_OK) return rc;
        if ((rc = check_view(k, d->k_stride, rows, d->T, d->Hk, d->Dk, es, &in[1], &vk, G)) != GDR_OK) return rc;
        if ((rc = check_view(v, d->v_stride, rows, d->T, d->Hk, d->Dv, es, &in[2], &vv, G)) != GDR_OK) return rc;
        if ((rc = check_view(d_o, d->do_stride, rows, d->T, d->H, d->Dv, es, &in[3], &vo, 1)) != GDR_OK) return rc;
        if (!dq || !dk || !dv) return GDR_E_NULL;
    }
    if (s.end > 0 && (!workspace || workspace_bytes < s.end)) return GDR_E_WORKSPACE;
    if (!g) return GDR_E_NULL;
    if (!aligned(g, 4) || !aligned(cu, 4) || !aligned(s0, 16) || !aligned(ds_final, 16) || !aligned(dq, 16) ||
        !aligned(dk, 16) || !aligned(dv, 16) || !aligned(dg, 4) || !aligned(ds0, 16) || !aligned(workspace, 16))
        return GDR_E_ALIGN;
    const size_t state = state_count(d) * 4, tokens = (size_t)rows * d->T;
    in[4] = range_of(g, (size_t)d->H * 4);
    in[5] = range_of(cu, ((size_t)d->B + 1) * 4);
    in[6] = range_of(s0, state);
    in[7] = range_of(ds_final, state);
    out[0] = range_of(dq, tokens * d->H * d->Dk * es);
    out[1] = range_of(dk, tokens * d->Hk * d->Dk * es);
    out[2] = range_of(dv, tokens * d->Hk * d->Dv * es);
    out[3] = range_of(dg, (size_t)d->H * 4);
    out[4] = range_of(ds0, state);
    out[5] = range_of(workspace, s.end);
    if (!alias_free(in, out)) return GDR_E_ALIAS;

    const hipStream_t st = static_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    auto at = [&](size_t off) { return reinterpret_cast<float *>(ws + off); };
    const size_t sums = sum_bytes(p);
    Walk wq, wv, wk;
    wq.a = vo; wq.b = vv; wq.c = vk;
    wq.Da = d->Dv; wq.Dc = d->Dk;
    wq.oscale = d->scale;
    wq.out = static_cast<char *>(dq);
    wq.e0 = s0; wq.e0_t = 1; wq.e0_decay = 1;
    wq.u = at(s.sums);
    wv.a = vk; wv.b = vq; wv.c = vo;
    wv.Da = d->Dk; wv.Dc = d->Dv;
    wv.reverse = 1;
    wv.uscale = d->scale;
    wv.out = shared ? ws + s.part_v : static_cast<char *>(dv);
    wv.out_f32 = shared;
    wv.e0 = ds_final;
    wv.ef = ds0;
    wv.u = at(s.sums + sums);
    wk.a = vv; wk.b = vo; wk.c = vq;
    wk.Da = d->Dv; wk.Dc = d->Dk;
    wk.reverse = 1;
    wk.uscale = d->scale;
    wk.out = shared ? ws + s.part_k : static_cast<char *>(dk);
    wk.out_f32 = shared;
    wk.e0 = ds_final; wk.e0_t = 1;
    wk.u = at(s.sums + 2 * sums);
    wv.u_t = wk.u;  // dv's and dk's states are transposes of each other: summed once
    wq.zero_outside = wv.zero_outside = wk.zero_outside = 1;
    const size_t groups = (size_t)p.b.units * d->H * p.slices;
    if (dg) {
        wq.x = vq;
        wk.x = vk;
        wq.chunk_e = wk.chunk_e = at(s.chunk_e);
        wq.dg_part = reinterpret_cast<double *>(ws + s.dg);
        wk.dg_part = wq.dg_part + groups;
    }
    WalkSet set;
    set.b = p.b;
    set.b.cu = cu;
    set.b.g = g;
    set.slices = p.slices;
    set.count = 2;
    set.w[0] = wq;
    set.w[1] = wv;
    set.w[2] = wk;
    if (p.sums && (rc = hip_status(gdr::hd::launch_segment_sums(set, bf16, p.sh, st))) != GDR_OK) return rc;
    set.count = 3;
    if (dg) {
        // dk's walk reads the states that dq's keeps
        set.count = 1;
        if ((rc = hip_status(gdr::hd::launch_walks(set, bf16, p.sh, true, st))) != GDR_OK) return rc;
        set.count = 2;
        set.w[0] = wk;
        if ((rc = hip_status(gdr::hd::launch_walks(set, bf16, p.sh, true, st))) != GDR_OK) return rc;
        if ((rc = hip_status(gdr::hd::launch_dg_sum(wq.dg_part, dg, p.b.units, d->H, p.slices, 2, groups, st))) != GDR_OK)
            return rc;
    } else {
        if ((rc = hip_status(gdr::hd::launch_walks(set, bf16, p.sh, false, st))) != GDR_OK) return rc;
    }
    if (shared) {
        const gdr::hd::GroupSum sk = {at(s.part_k), dk, tokens * d->Hk, d->Dk}, sv = {at(s.part_v), dv, tokens * d->Hk, d->Dv};
        return hip_status(gdr::hd::launch_group_sums(sk, sv, bf16, G, st));
    }
    return GDR_OK;
}

int gdr_head_decay_step(const gdr_head_decay_desc *d, const void *q, const void *k, const void *v, const float *g,
                        float *state, int32_t M, const int32_t *slots, const int32_t *parents, float *state_out,
                        void *o, void *stream) {
    int rc = check_desc(d, true);
    if (rc != GDR_OK) return rc;
    if (M < 0) return GDR_E_SHAPE;
    const bool in_place = !state_out || state_out == state, bf16 = d->dtype == GDR_BF16;
    if (in_place ? parents != nullptr : slots != nullptr) return GDR_E_MODE;
    if (!slots && !parents && (in_place ? M != d->B : M < d->B)) return GDR_E_SHAPE;
    if ((double)M * d->H * 65536.0 > (double)kMost || (double)d->B * d->H * 8 >= 2147483648.0) return GDR_E_SHAPE;
    if (d->B == 0 || d->H == 0) return GDR_OK;
    const int es = bf16 ? 2 : 4, G = d->H / d->Hk;
    gdr::hd::StepCall c;
    Range in[7] = {}, out[2] = {};
    if ((rc = check_view(q, d->q_stride, d->B, 1, d->H, d->Dk, es, &in[0], &c.q, 1)) != GDR_OK) return rc;
    if ((rc = check_view(k, d->k_stride, d->B, 1, d->Hk, d->Dk, es, &in[1], &c.k, G)) != GDR_OK) return rc;
    if ((rc = check_view(v, d->v_stride, d->B, 1, d->Hk, d->Dv, es, &in[2], &c.v, G)) != GDR_OK) return rc;
    if (!g || !o || (!state && M > 0)) return GDR_E_NULL;
    if (in_place && !state) return GDR_E_NULL;
    if (!aligned(g, 4) || !aligned(o, 16) || !aligned(state, 16) || !aligned(state_out, 16) || !aligned(slots, 4) ||
        !aligned(parents, 4))
        return GDR_E_ALIGN;
    const size_t one = (size_t)d->H * d->Dk * d->Dv * 4;
    in[3] = range_of(g, (size_t)d->H * 4);
    in[4] = range_of(slots, (size_t)d->B * 4);
    in[5] = range_of(parents, (size_t)d->B * 4);
    if (!in_place) in[6] = range_of(state, (size_t)M * one);
    out[0] = range_of(o, (size_t)d->B * d->H * d->Dv * es);
    out[1] = in_place ? range_of(state, (size_t)M * one) : range_of(state_out, (size_t)d->B * one);
    if (!alias_free(in, out)) return GDR_E_ALIAS;
    c.N = d->B;
    c.M = M;
    c.H = d->H;
    c.Dk = d->Dk;
    c.Dv = d->Dv;
    c.bf16 = bf16;
    c.scale = d->scale;
    c.g = g;
    c.state = state;
    c.slots = slots;
    c.parents = parents;
    c.state_out = in_place ? state : state_out;
    c.o = o;
    return hip_status(gdr::hd::launch_step(c, static_cast<hipStream_t>(stream)));
}

static int check_select(int32_t B, int32_t K, int32_t V) {
    if (B < 0 || K < 1 || V < 1) return GDR_E_SHAPE;
    if (K > gdr::beam::kMaxBeams || V > (1 << 30)) return GDR_E_UNSUPPORTED;
    if ((int64_t)K * V >= ((int64_t)1 << 31)) return GDR_E_SHAPE;
    // 64 parts of a row at most, four a workgroup
    if ((int64_t)B * K * 16 >= ((int64_t)1 << 31)) return GDR_E_SHAPE;
    return GDR_OK;
}

int gdr_beam_select_workspace_size(int32_t B, int32_t K, int32_t V, size_t *bytes) {
    if (!bytes) return GDR_E_NULL;
    const int rc = check_select(B, K, V);
    if (rc != GDR_OK) return rc;
    *bytes = gdr::beam::select_workspace_bytes(B, K, V);
    return GDR_OK;
}

int gdr_beam_select(int32_t B, int32_t K, int32_t V, int32_t dtype, const void *logits, int64_t row_stride,
                    const float *scores, const uint8_t *done, int32_t eos_token, int32_t pad_token, float *out_scores,
                    int32_t *out_tokens, int32_t *out_parents, uint8_t *out_done, void *workspace,
                    size_t workspace_bytes, void *stream) {
    const int rc = check_select(B, K, V);
    if (rc != GDR_OK) return rc;
    if (dtype != GDR_F32 && dtype != GDR_BF16) return GDR_E_MODE;
    if (pad_token < 0 || pad_token >= V) return GDR_E_MODE;
    const size_t es = dtype == GDR_BF16 ? 2 : 4, rows = (size_t)B * K;
    if (rows > 1 && row_stride < 0) return GDR_E_SHAPE;
    if (rows <= 1) row_stride = 0;
    if ((double)row_stride * (double)rows > (double)kMost) return GDR_E_SHAPE;
    if (B == 0) return GDR_OK;
    if (!logits || !scores || !out_scores || !out_tokens || !out_parents || !out_done) return GDR_E_NULL;
    const size_t need = gdr::beam::select_workspace_bytes(B, K, V);
    if (!workspace || workspace_bytes < need) return GDR_E_WORKSPACE;
    if (!aligned(logits, es) || !aligned(scores, 4) || !aligned(out_scores, 4) || !aligned(out_tokens, 4) ||
        !aligned(out_parents, 4) || !aligned(workspace, 16))
        return GDR_E_ALIGN;
    const Range in[] = {range_of(logits, ((rows - 1) * (size_t)row_stride + V) * es), range_of(scores, rows * 4),
                        range_of(done, rows)};
    const Range out[] = {range_of(out_scores, rows * 4), range_of(out_tokens, rows * 4),
                         range_of(out_parents, rows * 4), range_of(out_done, rows), range_of(workspace, need)};
    if (!alias_free(in, out)) return GDR_E_ALIAS;
    gdr::beam::SelectCall c;
    c.B = B;
    c.K = K;
    c.V = V;
    c.bf16 = dtype == GDR_BF16;
    c.logits = static_cast<const char *>(logits);
    c.row_stride = row_stride;
    c.scores = scores;
    c.done = done;
    c.eos = eos_token;
    c.pad = pad_token;
    c.out_scores = out_scores;
    c.out_tokens = out_tokens;
    c.out_parents = out_parents;
    c.out_done = out_done;
    c.ws = workspace;
    return hip_status(gdr::beam::launch_select(c, static_cast<hipStream_t>(stream)));
}

int gdr_beam_reorder(int32_t L, int32_t B, int32_t K, int64_t row_bytes, const void *state, const int32_t *parents,
                     void *out, void *stream) {
    if (L < 0 || B < 0 || K < 1 || row_bytes < 0) return GDR_E_SHAPE;
    if (K > gdr::beam::kMaxBeams) return GDR_E_UNSUPPORTED;
    if (row_bytes % 16) return GDR_E_ALIGN;
    if ((double)L * B * K * (double)row_bytes > 4.0 * (double)kMost) return GDR_E_SHAPE;
    if (L == 0 || B == 0 || row_bytes == 0) return GDR_OK;
    if (((double)row_bytes / 4096 + 1) * L * B >= 2147483648.0) return GDR_E_SHAPE;
    if (!state || !parents || !out) return GDR_E_NULL;
    if (!aligned(state, 16) || !aligned(out, 16) || !aligned(parents, 4)) return GDR_E_ALIGN;
    const size_t bytes = (size_t)L * B * K * row_bytes;
    const Range in[] = {range_of(parents, (size_t)B * K * 4), state == out ? range_of(nullptr, 0) : range_of(state, bytes)};
    const Range outs[] = {range_of(out, bytes)};
    if (!alias_free(in, outs)) return GDR_E_ALIAS;
    return hip_status(gdr::beam::launch_reorder(L, B, K, row_bytes, state, parents, out, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
