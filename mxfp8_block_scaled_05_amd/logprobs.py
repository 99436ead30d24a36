"""Token log-probabilities, entropy and top alternatives of logits, and their
gradient (include/mxfp8_tokens.h).

    r = token_logprobs(logits, targets, temperature=1.0, top_n=0)
    d = token_logprobs_backward(logits, targets, r.stats, r.entropy, d_logprobs, d_entropy)
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _check
from ._tokens import ERR_SHAPE, MAX_TOP, need, need_rows, same_device, stream_of, tokens_lib


@dataclass
class TokenLogprobs:
    logprobs: torch.Tensor                  # fp32 [T]: log p of the targets, 0 where there is none
    entropy: torch.Tensor                   # fp32 [T]
    stats: torch.Tensor                     # fp32 [T, 2]: max and log sum of exp(z - max), for the gradient
    top_logprobs: torch.Tensor | None       # fp32 [T, top_n]
    top_ids: torch.Tensor | None            # int64 [T, top_n]


def _logits_targets(logits, targets):
    code, ld = need_rows(logits, "logits")
    ids = need(targets, torch.int64, "targets")
    T, V = logits.shape
    if targets.numel() != T:
        raise ValueError("targets must have T = %d entries" % T)
    return code, ld, T, V, ids, same_device(logits, targets)


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, *, temperature: float = 1.0,
                   top_n: int = 0) -> TokenLogprobs:
    """Log-probability of ``targets`` (int64 [T]; outside [0, V): none, 0) under
    softmax(logits / temperature), the entropy, and the ``top_n`` (at most 64)
    likeliest columns with theirs, from one pass over logits (fp32 or bf16
    [T, V], rows contiguous, any row stride) (mxfp8_token_logprobs)."""
    code, ld, T, V, tg, dev = _logits_targets(logits, targets)
    L = tokens_lib()
    logprobs = logits.new_empty(T, dtype=torch.float32)
    entropy = torch.empty_like(logprobs)
    stats = logprobs.new_empty(T, 2)
    top = ids = None
    if top_n:
        if not 0 < top_n <= MAX_TOP:
            _check(ERR_SHAPE, "mxfp8_token_logprobs")
        top = logprobs.new_empty(T, top_n)
        ids = targets.new_empty(T, top_n)
    need_ws = L.mxfp8_token_logprobs_workspace_bytes(T, V, top_n)
    ws = logprobs.new_empty(need_ws // 4) if need_ws else None
    _check(L.mxfp8_token_logprobs(logits.data_ptr(), code, ld, T, V, tg, temperature, top_n, logprobs.data_ptr(),
                                  entropy.data_ptr(), stats.data_ptr(), top.data_ptr() if top_n else None,
                                  ids.data_ptr() if top_n else None, ws.data_ptr() if need_ws else None, need_ws,
                                  stream_of(dev)), "mxfp8_token_logprobs")
    return TokenLogprobs(logprobs, entropy, stats, top, ids)


def token_logprobs_backward(logits: torch.Tensor, targets: torch.Tensor, stats: torch.Tensor,
                            entropy: torch.Tensor | None, d_logprobs: torch.Tensor | None,
                            d_entropy: torch.Tensor | None = None, *, temperature: float = 1.0,
                            out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of token_logprobs' logprobs and entropy with respect to the
    logits, in their dtype (mxfp8_token_logprobs_backward).  Either gradient
    may be None.  ``out`` may be the logits themselves (in place), but share no
    memory with them otherwise."""
    code, ld, T, V, tg, dev = _logits_targets(logits, targets)
    if d_logprobs is None and d_entropy is None:
        raise ValueError("give d_logprobs, d_entropy or both")
    if d_entropy is not None and entropy is None:
        raise ValueError("d_entropy needs entropy")
    st = need(stats, torch.float32, "stats")
    if tuple(stats.shape) != (T, 2):
        raise ValueError("stats must be [T, 2]")
    rows = []
    for t, name in ((entropy, "entropy"), (d_logprobs, "d_logprobs"), (d_entropy, "d_entropy")):
        rows.append(None if t is None else need(t, torch.float32, name))
        if t is not None and t.numel() != T:
            raise ValueError("%s must have T = %d entries" % (name, T))
    same_device(logits, stats, entropy, d_logprobs, d_entropy)
    if out is None:
        out = logits.new_empty(T, V)
        ld_out = V
    else:
        out_code, ld_out = need_rows(out, "out")
        if out_code != code or tuple(out.shape) != (T, V):
            raise ValueError("out must be [T, V] in the logits' dtype")
        same_device(logits, out)
    _check(tokens_lib().mxfp8_token_logprobs_backward(logits.data_ptr(), code, ld, T, V, tg, st, *rows, temperature,
                                                      out.data_ptr(), ld_out, stream_of(dev)),
           "mxfp8_token_logprobs_backward")
    return out
