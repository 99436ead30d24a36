/*
 * mxfp8_tokens.h -- C ABI of the token-level operators around the MXFP8
 * layers: expert routing, the experts' row tables, expert rows back to
 * tokens, and token log-probabilities, each with its gradient.
 *
 * The expert GEMMs and gather quantizers of mxfp8.h read token rows sorted by
 * expert; these calls decide the experts, build those tables on the device
 * and bring the experts' outputs back.  A policy's update and its sampler
 * both need the log-probabilities of given tokens and the entropy of the
 * distribution they were drawn from.
 *
 * The conventions of mxfp8.h hold (row-major, caller-owned buffers, host
 * validation before anything is enqueued, one stream, no allocation, no
 * synchronization, graph-capturable, deterministic), except for alignment:
 * every pointer here needs only its element's own (2 bytes for bf16, 4 for
 * fp32 and int32, 8 for int64), MXFP8_ERR_ALIGN otherwise, so views that
 * start at any row or column are fine, and rows may lie any number of elements
 * apart (T * ld <= 2^60).  An output that shares memory with an input or with
 * another output is refused (MXFP8_ERR_OVERLAP) except where a call names it;
 * strided rows may lie between each other's.  Sums, softmax statistics and
 * gradients are computed in fp32 and rounded once on output.
 */
#ifndef MXFP8_TOKENS_H
#define MXFP8_TOKENS_H

#include "mxfp8.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MXFP8_SCORE_SOFTMAX = 0, MXFP8_SCORE_SIGMOID = 1 } mxfp8_score;

/*
 * mxfp8_route -- the experts of every token and their weights.
 *
 *   s = softmax(x) or sigmoid(x) over the E logits of a token
 *   c = s + bias (bias balances the choice only; NULL: c = s)
 *   groups > 1: the experts form `groups` runs of E / groups; a run's score
 *     is the sum of its group_top (1 or 2) largest c; the groups_kept best
 *     runs stay
 *   ids[t][0..k): the k largest c left, largest first
 *   weights[t][j] = s[ids[j]], over their sum if renormalize, times scale
 *
 * Equal values go to the lower index, for experts and for runs.  The choice
 * is that of scores held in fp64 (scores closer than fp32 can tell apart are
 * compared again in fp64); without a bias (and with group_top 1, if there are
 * groups) it is that of the logits, which the scores rise with.
 *
 * A logit of -Inf has score 0.  Renormalized weights hold however small the
 * chosen scores are; they are NaN if no chosen logit is above -Inf, and all
 * softmax weights are if no logit is, or if one is +Inf.  With a NaN among the
 * logits the ids are k distinct experts and the weights NaN (sigmoid: those of
 * the NaN experts, all if renormalized).
 *
 *   logits : [T][E] FP32 or BF16, rows ld >= E elements apart
 *   bias   : FP32 [E] or NULL
 *   ids    : int32 [T][k];  weights: FP32 [T][k]
 * T >= 0 (0 enqueues nothing), 1 <= E <= 512, 1 <= k <= 32, 1 <= groups <=
 * 64, E % groups == 0, 1 <= groups_kept <= groups, k <= groups_kept * E /
 * groups, group_top <= E / groups, T < 2^26.  MXFP8_ERR_DTYPE for an unknown
 * dtype or score.
 */
mxfp8_status mxfp8_route(const void *logits, mxfp8_dtype dtype, int64_t ld, int64_t T, int64_t E, int64_t k,
                         mxfp8_score score, const float *bias, int64_t groups, int64_t groups_kept,
                         int64_t group_top, int renormalize, float scale, int32_t *ids, float *weights,
                         hipStream_t stream);

/*
 * mxfp8_route_backward -- gradient of the weights with respect to the logits
 * (the choice itself has none, nor has the bias).
 *
 *   d_logits [T][E] in the logits' dtype, all of it written; ids as
 *   mxfp8_route gives them (distinct within a token; an id outside [0, E) is
 *   no expert).  Limits as mxfp8_route's.
 */
mxfp8_status mxfp8_route_backward(const void *logits, mxfp8_dtype dtype, int64_t ld, int64_t T, int64_t E,
                                  int64_t k, mxfp8_score score, const int32_t *ids, const float *d_weights,
                                  int renormalize, float scale, void *d_logits, hipStream_t stream);

/* Rows that the padded expert groups of `pairs` (token, expert) pairs over E
 * experts can take at most: the size of mxfp8_route_tables' row_token and of
 * the expert-sorted matrices.  Pure host function; 0 for invalid sizes. */
int64_t mxfp8_route_rows(int64_t pairs, int64_t E, int64_t pad);

/* Workspace bytes of mxfp8_route_tables (0: none needed, or invalid sizes). */
size_t mxfp8_route_tables_workspace_bytes(int64_t T, int64_t k, int64_t E);

/*
 * mxfp8_route_tables -- expert ids of every token -> the row tables of the
 * expert-sorted, padded layout.
 *
 * The pairs (t, j) are sorted by expert and then by pair index; expert e's
 * rows start at offsets[e] and its group is padded to a multiple of `pad`
 * rows (32: the grouped GEMMs' groups; 128: the weight gradients').
 *   offsets   : int32 [E+1], the d_group_offsets of the grouped GEMMs
 *   counts    : int32 [E], rows of each expert without padding
 *   row_token : int64 [rows], the token of each row, -1 for padding rows and
 *               for those from offsets[E] on (d_row_index of the gather
 *               quantizers)
 *   pair_row  : int32 [T][k], the row of each pair, -1 for an id outside
 *               [0, E) (a token without an expert there)
 * rows >= mxfp8_route_rows(T * k, E, pad) (MXFP8_ERR_SHAPE if less).
 *   workspace : mxfp8_route_tables_workspace_bytes(T, k, E) bytes, 4-byte
 *               aligned, NULL if that is 0; MXFP8_ERR_SHAPE if
 *               workspace_bytes is less.
 * T, k >= 1, 1 <= E <= 1024, 1 <= pad <= 1024, T * k + E * pad < 2^31.
 */
mxfp8_status mxfp8_route_tables(const int32_t *ids, int64_t T, int64_t k, int64_t E, int64_t pad,
                                int32_t *offsets, int32_t *counts, int64_t *row_token, int64_t rows,
                                int32_t *pair_row, void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * mxfp8_moe_combine -- out[t] = sum_j weights[t][j] * y[pair_row[t][j]], added
 * in the order of j.  y [rows][H] and out [T][H] FP32 or BF16; a pair_row
 * outside [0, rows) adds nothing (a token with no rows gets zeros).
 * T, rows >= 0 (T = 0 enqueues nothing), H, k >= 1, T * k + rows / 8 < 2^26,
 * T * ceil(H / 4) < 2^31, rows * H <= 2^60.
 */
mxfp8_status mxfp8_moe_combine(const void *y, mxfp8_dtype dtype, int64_t rows, int64_t H, const int32_t *pair_row,
                               const float *weights, int64_t T, int64_t k, void *out, hipStream_t stream);

/*
 * mxfp8_moe_combine_backward -- gradients of mxfp8_moe_combine.
 *   d_y [rows][H] in y's dtype: weights[t][j] * d_out[t] in row
 *     pair_row[t][j], zeros where row_token is outside [0, T) (padding)
 *   d_weights FP32 [T][k]: <d_out[t], y[pair_row[t][j]]>, 0 where pair_row is
 *     outside [0, rows)
 * pair_row and row_token are one mxfp8_route_tables result: each row belongs
 * to one pair or to none (rows of other tables are left unspecified, never
 * addressed outside the buffers).  d_y may be y and d_weights the weights
 * (same pointers).  Limits as mxfp8_moe_combine's.
 */
mxfp8_status mxfp8_moe_combine_backward(const void *d_out, const void *y, mxfp8_dtype dtype, int64_t rows, int64_t H,
                                        const int32_t *pair_row, const float *weights, const int64_t *row_token,
                                        int64_t T, int64_t k, void *d_y, float *d_weights, hipStream_t stream);

/* Workspace bytes with which mxfp8_token_logprobs splits its rows over the
 * current device (0: it would not split; also 0 for invalid sizes). */
size_t mxfp8_token_logprobs_workspace_bytes(int64_t T, int64_t V, int64_t top_n);

/*
 * mxfp8_token_logprobs -- log-probabilities of given tokens, entropy, and the
 * likeliest tokens, from one pass over the logits.
 *
 *   z = x / temperature, m = max z, L = log sum e^(z - m), log p = z - m - L
 *   logprobs[t] = log p[targets[t]], 0 for a target outside [0, V)
 *   entropy[t]  = -sum p log p (terms with p = 0 are 0)
 *   stats[t]    = (m, L), what the gradient needs: m rounded to fp32 (finite
 *     logits: to a finite number) and, while |m| < 2^31, L to that m
 *   top_ids[t][0..top_n), top_logprobs: the columns of the largest logits,
 *     largest first, the lower column first among equals, and their log p
 * Logits of -Inf are tokens that cannot occur; a row of nothing else has
 * m = -Inf and NaN for the rest, as has a row with a NaN or +Inf in it (its
 * top_ids are columns all the same).
 *
 *   logits  : [T][V] FP32 or BF16, rows ld >= V elements apart
 *   targets : int64 [T];  logprobs, entropy: FP32 [T];  stats: FP32 [T][2]
 *   top_logprobs, top_ids: FP32 / int64 [T][top_n], NULL if top_n is 0
 *   workspace: 16-byte aligned or NULL; with at least
 *     mxfp8_token_logprobs_workspace_bytes(T, V, top_n) bytes, few rows are
 *     split over more workgroups (results differ from the unsplit call's in
 *     the order of the sums only).
 * T >= 0 (0 enqueues nothing), 1 <= V < 2^31, 0 <= top_n <= min(V, 64),
 * 2^-60 <= temperature <= 2^60, T * ceil(V / 4096) < 2^24.
 */
mxfp8_status mxfp8_token_logprobs(const void *logits, mxfp8_dtype dtype, int64_t ld, int64_t T, int64_t V,
                                  const int64_t *targets, double temperature, int64_t top_n, float *logprobs,
                                  float *entropy, float *stats, float *top_logprobs, int64_t *top_ids,
                                  void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * mxfp8_token_logprobs_backward -- gradient of log-probability and entropy.
 *
 *   d_logits[t][v] = (g (1[v = target] - p) - h p (log p + entropy)) /
 *   temperature, g = d_logprobs[t] (0 where the target is outside [0, V)),
 *   h = d_entropy[t]; a term whose gradient is NULL is left out (not both;
 *   entropy may be NULL with d_entropy).  Columns of -Inf get 0 (the
 *   target's g / temperature).  A row whose L is NaN (a NaN or +Inf among its
 *   logits, or nothing above -Inf) gets NaN in every column, whatever g and h
 *   are.  Where |m| >= 2^31, logits whose z rounds to m in fp32 have p = e^-L
 *   and the others 0 (rows of the type's lowest value: the same p for all).
 *   stats and entropy as mxfp8_token_logprobs gave them for the same logits
 *   and temperature.  d_logits: rows ld_out >= V apart, in the logits' dtype;
 *   it may be the logits themselves (same pointer and ld).
 */
mxfp8_status mxfp8_token_logprobs_backward(const void *logits, mxfp8_dtype dtype, int64_t ld, int64_t T, int64_t V,
                                           const int64_t *targets, const float *stats, const float *entropy,
                                           const float *d_logprobs, const float *d_entropy, double temperature,
                                           void *d_logits, int64_t ld_out, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP8_TOKENS_H */
