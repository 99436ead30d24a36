/*
 * mxfp8_policy.h -- C ABI of the operators that a policy trained and sampled
 * with low-rank adapters needs around the MXFP8 layers: the gated activation
 * with its inputs kept in 8 bits for the backward pass.
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

#ifdef __cplusplus
}
#endif

#endif /* MXFP8_POLICY_H */
