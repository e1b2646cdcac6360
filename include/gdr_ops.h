/*
 * gdr_ops.h -- C ABI of libgdr: linear attention with one decay per head, and
 * beam search over decode steps.  Status codes, dtypes and the conventions for
 * every entry point are those of gdr.h (device pointers owned by the caller,
 * nothing allocated, nothing synchronised, every argument checked on the host
 * before any HIP call, GDR_OK = enqueued on `stream`).
 *
 * Linear attention with a decay per head.  For each sequence and query head h
 * with lambda = exp(g[h]) (lambda^0 = 1 also for g = -inf), key/value head
 * h / (H / Hk), and the fp32 state S (Dk x Dv):
 *
 *   S_t = lambda S_{t-1} + k_t v_t^T        o_t = scale * S_t^T q_t
 *
 * It is the additive write of gdr.h (GDR_DELTA_OFF) with a decay that does not
 * depend on the token: no gate tensor is read, the factors of a chunk are the
 * same for all chunks, and there is nothing to solve.
 *
 * Layouts of this family:
 *  - q [.., H, Dk], k [.., Hk, Dk], v [.., Hk, Dv] and d_o [.., H, Dv] may be
 *    strided: the last dimension is contiguous, the others have the strides of
 *    the descriptor (in elements, >= 0; 0 repeats a row; between tokens 16 MiB
 *    at most), with every row 16-byte aligned.  Views of one fused projection need no copy.
 *  - Outputs and states are contiguous; dq, dk, dv have the inputs' type.
 *  - Hk divides H, H is at most 16384; Dk and Dv are multiples of 8 from 8 to 256.
 *  - Values are not checked: g should be <= 0.  A value of k, v or d_o that is not
 *    finite makes the other tokens of its chunk (64 tokens at most, also
 *    earlier ones) undefined, not only the later ones;
 *    so does a state that is not finite for all of its outputs.
 */
#ifndef GDR_OPS_H
#define GDR_OPS_H

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gdr_head_decay_desc {
    int32_t B;      /* sequences */
    int32_t T;      /* tokens per sequence (packed: tokens in all); ignored by the step */
    int32_t H;      /* query heads */
    int32_t Hk;     /* key/value heads, a divisor of H */
    int32_t Dk;     /* key width */
    int32_t Dv;     /* value width */
    int32_t dtype;  /* GDR_F32 or GDR_BF16: q, k, v, o, d_o, dq, dk, dv */
    float scale;    /* output scale */
    int64_t q_stride[3];   /* elements between sequences (not read when packed), */
    int64_t k_stride[3];   /*   tokens (not read by the step), heads             */
    int64_t v_stride[3];
    int64_t do_stride[3];  /* backward only */
} gdr_head_decay_desc;

/*
 * Whole sequences (prefill, training's forward pass).
 *   q, k, v    strided, see above
 *   g          [H] fp32 log-decays
 *   s0         [B, H, Dk, Dv] fp32, or NULL for zero
 *   o          [B, T, H, Dv] (written)
 *   s_final    [B, H, Dk, Dv] fp32 (written), or NULL; may equal s0
 *   cu_seqlens NULL: B sequences of T tokens.  Else a packed batch: [B + 1] int32
 *              in device memory, sequence n holds tokens [cu[n], cu[n+1]) of the
 *              T tokens; entries are clamped to [0, T] and raised to the
 *              largest before them, rows of o outside every sequence are left
 *              as they were.
 *   workspace  at least the queried bytes, 16-byte aligned; `packed` as the call
 *              that follows.  NULL is allowed where the query gives 0.
 */
int gdr_head_decay_fwd_workspace_size(const gdr_head_decay_desc *desc, int packed, size_t *bytes);
int gdr_head_decay_fwd(const gdr_head_decay_desc *desc, const int32_t *cu_seqlens,
                       const void *q, const void *k, const void *v, const float *g,
                       const float *s0, void *o, float *s_final,
                       void *workspace, size_t workspace_bytes, void *stream);

/*
 * Its backward pass.
 *   d_o       [B, T, H, Dv] dL/do, strided, the inputs' type
 *   ds_final  [B, H, Dk, Dv] fp32 dL/ds_final, or NULL for zero
 *   dq        [B, T, H, Dk], dk [B, T, Hk, Dk], dv [B, T, Hk, Dv] (written; dk
 *             and dv summed over the query heads that share them).  In a packed
 *             batch the rows outside every sequence are set to zero.
 *   dg        [H] fp32 dL/dg (written), or NULL: without it the states of the
 *             chunks are not kept
 *   ds0       [B, H, Dk, Dv] fp32 (written), or NULL
 * Sums run in a fixed order: equal calls give equal bits.
 */
int gdr_head_decay_bwd_workspace_size(const gdr_head_decay_desc *desc, int packed, int need_dg,
                                      size_t *bytes);
int gdr_head_decay_bwd(const gdr_head_decay_desc *desc, const int32_t *cu_seqlens,
                       const void *q, const void *k, const void *v, const float *g,
                       const float *s0, const void *d_o, const float *ds_final,
                       void *dq, void *dk, void *dv, float *dg, float *ds0,
                       void *workspace, size_t workspace_bytes, void *stream);

/*
 * One token for each of B sequences (decode): q [B, H, Dk], k [B, Hk, Dk],
 * v [B, Hk, Dv] strided (sequence, -, head), o [B, H, Dv] (written).
 *   state      [M, H, Dk, Dv] fp32
 *   state_out  NULL or equal to state: the states are updated in place, and M
 *              must be B unless slots are given.  Otherwise [B, H, Dk, Dv]:
 *              row n continues from state[n], or from state[parents[n]], and
 *              writes state_out[n]; state is only read.
 *   slots      (in place only) [B] int32, row n works on state[slots[n]].  A slot
 *              outside [0, M) marks a padded row: its o is zero, no state is
 *              touched.  Where a slot is named twice the lowest row has it and
 *              the others are padded rows.
 *   parents    (with state_out only) [B] int32; parents may repeat (the beams of
 *              a search that continue from one state); outside [0, M) the row
 *              starts from a zero state.
 */
int gdr_head_decay_step(const gdr_head_decay_desc *desc,
                        const void *q, const void *k, const void *v, const float *g,
                        float *state, int32_t M, const int32_t *slots, const int32_t *parents,
                        float *state_out, void *o, void *stream);

/*
 * Beam search, one step's selection for B requests of K beams over V tokens:
 *   cand(k, v) = scores[b, k] + logits[b, k, v] - logsumexp_v logits[b, k, :]
 * with a candidate that is not a finite number counting as -inf, and a beam that
 * is done offering pad_token at its own score and nothing else (-inf).  The K
 * best candidates, best first, equal ones by the lowest k V + v, are returned
 * as score, token and parent; done' = done[parent] or token == eos_token.
 * Candidates are compared in fp64 (the log-sum is of fp32 exponentials summed
 * in fp64).
 *   logits  [B, K, V] GDR_F32 or GDR_BF16, rows `row_stride` elements apart (a
 *           request's K rows, then the next request's); any element alignment
 *   scores  [B, K] fp32; done [B, K] bytes (0 or 1), or NULL: none
 *   out_*   scores fp32, tokens int32, parents int32, done bytes, all [B, K]
 * 1 <= K <= 32, 1 <= V <= 2^30, K V < 2^31, 0 <= pad_token < V; eos_token outside [0, V):
 * no beam ends here.  Outputs must not overlap inputs.
 */
int gdr_beam_select_workspace_size(int32_t B, int32_t K, int32_t V, size_t *bytes);
int gdr_beam_select(int32_t B, int32_t K, int32_t V, int32_t dtype, const void *logits,
                    int64_t row_stride, const float *scores, const uint8_t *done,
                    int32_t eos_token, int32_t pad_token, float *out_scores, int32_t *out_tokens,
                    int32_t *out_parents, uint8_t *out_done, void *workspace,
                    size_t workspace_bytes, void *stream);

/*
 * Reordering of the states of a search: new[l, b, k] = old[l, b, parents[b, k]]
 * for L x B x K rows of row_bytes (a multiple of 16) bytes each.
 *   out == state: in place; only rows whose parent is another row move, each
 *   parent is read once.  Otherwise every row is written to out.
 *   parents [B, K] int32 in device memory; outside [0, K) a row keeps its state.
 * 1 <= K <= 32; state and out 16-byte aligned and equal or not overlapping.
 */
int gdr_beam_reorder(int32_t L, int32_t B, int32_t K, int64_t row_bytes, const void *state,
                     const int32_t *parents, void *out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_OPS_H */
