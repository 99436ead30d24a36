"""Verification of drafted tokens against the target's probabilities
(include/mxfp8_policy.h).

    r = verify_drafts(logits, offsets, draft_ids, uniforms, noise, draft_logits=q_logits, temperature=0.7)
    r.accepted, r.tokens, r.logprobs
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _check
from ._policy import ERR_SHAPE, need, need_rows, policy_lib, same_device, stream_of


@dataclass
class DraftVerdict:
    accepted: torch.Tensor          # int32 [B]: drafted tokens of each request that stand
    tokens: torch.Tensor            # int64 [R], by row of the logits: those, the next token, then -1
    logprobs: torch.Tensor          # fp32 [R]: log p of these tokens, 0 behind them


def verify_drafts(logits: torch.Tensor, offsets: torch.Tensor, draft_ids: torch.Tensor, uniforms: torch.Tensor,
                  noise: torch.Tensor, *, draft_logits: torch.Tensor | None = None,
                  temperature: float = 1.0) -> DraftVerdict:
    """Which drafted tokens of each request stand and the token after them, so
    that what comes out is distributed as softmax(logits / temperature)
    (mxfp8_verify_drafts).

    logits fp32 or bf16 [R, V] (rows contiguous, any row stride): request b has
    rows offsets[b] to offsets[b + 1] (int32 [B + 1], on the device), one for
    each drafted token and one after the last.  draft_ids int64, uniforms fp32 in
    [0, 1), both [R - B], and draft_logits [R - B, V] in the logits' dtype, what
    the tokens were drawn from (None: they were looked up), are in the same order
    without the last rows.  noise fp32 [B, V]: exponential draws (rate 1), as
    torch.Tensor.exponential_ gives them."""
    code, ld = need_rows(logits, "logits")
    R, V = logits.shape
    po = need(offsets, torch.int32, "offsets")
    B = offsets.numel() - 1
    if B < 0 or R < B or (B == 0 and R):
        raise ValueError("offsets must be [B + 1] with a row at least for each request, got %d for R = %d rows" % (B + 1, R))
    D = R - B
    ids, u = need(draft_ids, torch.int64, "draft_ids"), need(uniforms, torch.float32, "uniforms")
    if draft_ids.numel() != D or uniforms.numel() != D:
        raise ValueError("draft_ids and uniforms must have R - B = %d entries" % D)
    noise_code, ld_noise = need_rows(noise, "noise")
    if noise.dtype is not torch.float32 or tuple(noise.shape) != (B, V):
        raise ValueError("noise must be fp32 [B = %d, V = %d]" % (B, V))
    pd, ld_draft = None, V
    if draft_logits is not None:
        draft_code, ld_draft = need_rows(draft_logits, "draft_logits")
        if draft_code != code or tuple(draft_logits.shape) != (D, V):
            raise ValueError("draft_logits must be [R - B = %d, V = %d] in the logits' dtype" % (D, V))
        pd = draft_logits.data_ptr() if D else None
    dev = same_device(logits, offsets, draft_ids, uniforms, noise, draft_logits)
    L = policy_lib()
    need_ws = L.mxfp8_verify_drafts_workspace_bytes(R, B, V, pd is not None)
    if not need_ws and B:
        _check(ERR_SHAPE, "mxfp8_verify_drafts")
    ws = noise.new_empty(need_ws // 4)
    accepted, tokens = offsets.new_empty(B), draft_ids.new_empty(R)
    logprobs = noise.new_empty(R)
    _check(L.mxfp8_verify_drafts(logits.data_ptr(), code, ld, R, V, po, B, ids, u, pd, ld_draft, noise.data_ptr(), ld_noise,
                                 temperature, accepted.data_ptr(), tokens.data_ptr(), logprobs.data_ptr(), ws.data_ptr(),
                                 need_ws, stream_of(dev)), "mxfp8_verify_drafts")
    return DraftVerdict(accepted, tokens, logprobs)
