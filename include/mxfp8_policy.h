/*
 * mxfp8_policy.h -- C ABI of the operators that a policy trained and sampled
 * with low-rank adapters needs around the MXFP8 layers: the gated activation
 * with its inputs kept in 8 bits for the backward pass, the adapters beside a
 * shared projection with their gradients, and the verification of drafted
 * tokens.
 *
 * The conventions of mxfp8.h hold (row-major, caller-owned buffers, host
 * validation before anything is enqueued, one stream, no allocation, no
 * synchronization, graph-capturable, deterministic).  Every output that shares
 * memory with an input or with another output is refused (MXFP8_ERR_OVERLAP)
 * except where a call names it.  Workspaces are read and written by the call's
 * own kernels only; what they hold before it does not matter, and two calls
 * that may run at once need one each.
 */
#ifndef MXFP8_POLICY_H
#define MXFP8_POLICY_H

#include "mxfp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * mxfp8_swiglu -- h = silu(gate) * up, with gate and up kept as MXFP8.
 *
 *   gu : BF16 [T][2 I], rows ld >= 2 I elements apart: gate in columns
 *        [0, I), up in [I, 2 I)
 *   h  : silu(g) u = g u / (1 + e^-g) in fp32, rounded once to BF16, then
 *     h_bf16 given        : [T][I]
 *     h_q and h_s given   : exactly what mxfp8_quantize(h, axis 1) writes for
 *       it ([T][I] and [T][I/32]; h_layout MXFP8_CANONICAL), or what
 *       mxfp8_repack writes for that grid (MXFP8_PACKED: N = T, K = I, padding
 *       included), the operand of the next projection
 *     (one of the two)
 *   saved_q, saved_s : the checkpoint, both or neither: exactly
 *     mxfp8_quantize(gu, axis 1), [T][2 I] and [T][2 I / 32]; 2.06 bytes an
 *     element of h instead of 4
 *
 * T >= 0 (0 enqueues nothing), I >= 32, I % 32 == 0, ld % 8 == 0, T * I < 2^35
 * and, packed, the limits of mxfp8_repack; all pointers 16-byte aligned.
 */
mxfp8_status mxfp8_swiglu(const void *gu_bf16, int64_t ld, int64_t T, int64_t I, void *h_bf16, uint8_t *h_q,
                          uint8_t *h_s, mxfp8_layout h_layout, uint8_t *saved_q, uint8_t *saved_s,
                          hipStream_t stream);

/*
 * mxfp8_swiglu_backward -- its gradient from the checkpoint.
 *
 *   g, u = the checkpoint's values; s = 1 / (1 + e^-g)
 *   d_gu [T][2 I] BF16: d_g = d_h u s (1 + g (1 - s)), d_u = d_h g s
 *   h_bf16 [T][I] or NULL: g s u again, from the checkpoint's values (the next
 *     projection's weight gradient needs it along tokens; keeping it from the
 *     forward pass would cost 2 bytes an element)
 *   d_h : BF16 [T][I], rows ld >= I elements apart
 * Computed in fp32, rounded once.  A block of the checkpoint that held a NaN
 * or Inf is NaN in all its 32 columns (as mxfp8_dequantize gives it).
 * Limits as mxfp8_swiglu's; h_bf16 may be d_h (same pointer, ld == I).
 */
mxfp8_status mxfp8_swiglu_backward(const void *d_h_bf16, int64_t ld, int64_t T, int64_t I, const uint8_t *saved_q,
                                   const uint8_t *saved_s, void *d_gu_bf16, void *h_bf16, hipStream_t stream);

/*
 * Low-rank adapters of many requests beside a shared projection.
 *
 * Row t of a batch belongs to adapter e (or to none); adapter e adds
 *   scales[e] * B_e (A_e x_t)
 * to the shared projection's output y_t.  The rows come through the row tables
 * of mxfp8_route_tables, built with k = 1, the adapters as experts and pad a
 * multiple of 32 (once for all the layers of a batch):
 *   offsets   : DEVICE int32 [E+1], every entry a multiple of 32
 *   row_token : DEVICE int64 [rows], rows % 32 == 0: the row t of each sorted
 *               row, outside [0, T) for padding (it then adds nothing); rows
 *               from offsets[E] on are padding whatever they hold
 * Entries of offsets are clamped to [0, rows]; a row t named twice gets one of
 * its sums.  Malformed tables can give wrong sums, never an access outside the
 * buffers.
 *
 *   x : BF16 [T][K], rows ld_x elements apart
 *   a : BF16 [E][r][K];  b : BF16 [E][N][r];  scales : FP32 [E] or NULL (all 1)
 *   hidden : FP32 [rows][r], A_e x_t of every sorted row (zeros in padding)
 *
 * Common limits: 1 <= E <= 1024, 8 <= r <= 128 and r % 8 == 0 (pad a smaller
 * rank with zeros), K, N >= 8, K % 8 == 0, N % 8 == 0, strides % 8 == 0, 0 <=
 * T < 2^31, 0 <= rows < 2^31, T * stride <= 2^60, rows / 32 * ceil(max(K,
 * N) / 256) < 2^24, (rows / 256 + E) * ceil((K + N) / 128) < 2^22, E * r * (K +
 * N) < 2^40; all pointers 16-byte aligned but offsets and scales (4) and row_token (8).  T = 0: every row is padding.
 * The adapters' sums are held in fp32; A x and S enter the next product as sums
 * of BF16 numbers that keep all 24 bits where the result is FP32, 16 where it
 * is BF16.  An infinity among the operands, and a product that leaves FP32's
 * range, give the infinity or NaN that the formula gives.
 */

/* Workspace bytes of mxfp8_lora_add (0 for invalid sizes). */
size_t mxfp8_lora_add_workspace_bytes(int64_t rows, int64_t E, int64_t r, int64_t K, int64_t N);

/*
 * mxfp8_lora_add -- y += the adapters' products, in place.
 *   y : [T][N] FP32 or BF16, rows ld_y >= N elements apart; rows without an
 *       adapter are left as they are
 *   hidden : or NULL; kept for mxfp8_lora_backward
 *   workspace : mxfp8_lora_add_workspace_bytes(..) bytes, 16-byte aligned
 */
mxfp8_status mxfp8_lora_add(void *y, mxfp8_dtype y_dtype, int64_t ld_y, const void *x_bf16, int64_t ld_x, int64_t T,
                            const void *a_bf16, const void *b_bf16, const float *scales, int64_t E, int64_t r,
                            int64_t K, int64_t N, const int32_t *offsets, const int64_t *row_token, int64_t rows,
                            float *hidden, void *workspace, size_t workspace_bytes, hipStream_t stream);

/* The forms of mxfp8_lora_backward's x. */
typedef enum { MXFP8_INPUT_BF16 = 0, MXFP8_INPUT_CANONICAL = 1, MXFP8_INPUT_PACKED = 2 } mxfp8_input;

/* Workspace bytes of mxfp8_lora_backward (0 for invalid sizes). */
size_t mxfp8_lora_backward_workspace_bytes(int64_t rows, int64_t E, int64_t r, int64_t K, int64_t N);

/*
 * mxfp8_lora_backward -- gradients of mxfp8_lora_add.
 *
 *   S_t  = scales[e] * B_e^T d_y_t
 *   d_x += A_e^T S_t, in place: BF16 [T][K], rows ld_dx apart, the gradient
 *          that the shared projection's own product wrote before; NULL: left out
 *   d_a  = sum_t S_t x_t^T : FP32 [E][r][K];  d_b = sum_t scales[e] d_y_t
 *          hidden_t^T : FP32 [E][N][r]; all of both is written, zeros for an
 *          adapter without rows
 *   d_y : BF16 [T][N], rows ld_dy apart;  hidden as mxfp8_lora_add gave it
 *   x   : MXFP8_INPUT_BF16: BF16 [T][K], rows ld_x apart, x_s NULL
 *         MXFP8_INPUT_CANONICAL: mxfp8_quantize(x, axis 1)'s grid in x and x_s
 *           (K % 32 == 0; ld_x is not read): the input kept in 8 bits
 *         MXFP8_INPUT_PACKED: the same in mxfp8_repack's layout (N = T), the
 *           operand that the shared projection itself read
 *   workspace : mxfp8_lora_backward_workspace_bytes(..) bytes, 16-byte aligned
 * The sums over rows are cut at places that follow from the sizes alone and
 * joined in order.
 */
mxfp8_status mxfp8_lora_backward(void *d_x_bf16, int64_t ld_dx, const void *d_y_bf16, int64_t ld_dy, const void *x,
                                 const uint8_t *x_s, mxfp8_input x_input, int64_t ld_x, int64_t T,
                                 const void *a_bf16, const void *b_bf16, const float *scales, int64_t E, int64_t r, int64_t K, int64_t N,
                                 const int32_t *offsets, const int64_t *row_token, int64_t rows, const float *hidden,
                                 float *d_a, float *d_b, void *workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/* Workspace bytes of mxfp8_verify_drafts, with or without draft logits (0 for
 * invalid sizes). */
size_t mxfp8_verify_drafts_workspace_bytes(int64_t R, int64_t B, int64_t V, int draft_logits);

/*
 * mxfp8_verify_drafts -- which drafted tokens of each request stand, and the
 * token that follows them, from given random numbers; the tokens that come out
 * are distributed as if the target had been sampled.
 *
 * Request b has the rows [offsets[b], offsets[b+1]) of the target's logits: one
 * for each of its n drafted tokens, in order, and one after the last.  With
 * p = softmax(logits / temperature) of a row, q = softmax(draft_logits /
 * temperature) of the drafted token's row (1 at the token itself where
 * draft_logits is NULL: a draft that was looked up, not drawn), x the drafted
 * token and u its uniform:
 *   the drafted tokens stand up to the first with  not (u q(x) < p(x));
 *   the next token is the column with the largest w / noise, lowest first, of
 *     w = max(p - q, 0) at that position, or of w = p after the last draft;
 *     columns with w / noise not above 0 are not drawn
 * noise holds exponential draws (rate 1), so the column is drawn with
 * probability w / sum w.  Where p exceeds q nowhere (rounding, or a draft row
 * without a distribution), w = p.  The decisions are those of probabilities
 * held in fp64 (close ones are taken again in fp64), with noise of 2^-32 to
 * 2^32; a request with a close one, and every request of more than 31 drafted
 * tokens, takes several times as long.  A temperature near 0 (2^-60) with draft_logits NULL compares with the
 * largest logit: greedy verification.
 *
 *   accepted [B] int32 : drafted tokens that stand
 *   tokens   [R] int64 : by row: the drafted tokens that stand, the next one,
 *     then -1
 *   logprobs [R] FP32  : log p of those tokens, within 2^-16 and FP32's rounding;
 *     0 behind them
 * A row without a distribution (a NaN or +Inf in it, or nothing above -Inf)
 * lets no draft stand and gives no token: -1, log-probability NaN.  A drafted
 * token outside [0, V) does not stand.
 *
 *   logits : FP32 or BF16 [R][V], rows ld apart; draft_logits : the same dtype
 *     [R - B][V], rows ld_draft apart, or NULL; row offsets[b] - b + i is that
 *     of request b's i-th drafted token, as for
 *   draft_ids int64 [R - B], uniforms FP32 [R - B] in [0, 1)
 *   noise : FP32 [B][V], rows ld_noise apart
 *   offsets : DEVICE int32 [B+1], rising by at least 1, offsets[0] == 0,
 *     offsets[B] == R.  Entries are clamped to [0, R]; a request without rows
 *     has accepted 0 and no token; rows of no request are not written
 *   workspace : mxfp8_verify_drafts_workspace_bytes(..) bytes, 16-byte aligned
 * B >= 0 (0 enqueues nothing), B <= R < 2^31, 1 <= V < 2^31, 2^-60 <= temperature
 * <= 2^60, (2 R - B) * ceil(V / 4096) < 2^22; pointers aligned as their elements.
 */
mxfp8_status mxfp8_verify_drafts(const void *logits, mxfp8_dtype dtype, int64_t ld, int64_t R, int64_t V,
                                 const int32_t *offsets, int64_t B, const int64_t *draft_ids, const float *uniforms,
                                 const void *draft_logits, int64_t ld_draft, const float *noise, int64_t ld_noise,
                                 double temperature, int32_t *accepted, int64_t *tokens, float *logprobs,
                                 void *workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP8_POLICY_H */
