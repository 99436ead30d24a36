"""Expert routing around the grouped GEMMs (include/mxfp8_tokens.h).

    ids, w  = route(logits, k, ...)                  # experts of every token
    t       = route_tables(ids, E)                   # RouteTables: offsets, counts, row_token, pair_row
    ...       quantize_gather*(x, t.row_token), grouped_gemm*(.., t.offsets) -> y
    out     = moe_combine(y, t.pair_row, w)          # back in token order
    dy, dw  = moe_combine_backward(d_out, y, t.pair_row, w, t.row_token)
    dlogits = route_backward(logits, ids, dw, ...)
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _check, _need, _ptr, _stream
from ._tokens import need_rows, same_device, tokens_lib

_SCORES = {"softmax": 0, "sigmoid": 1}


def _score_code(score: str) -> int:
    code = _SCORES.get(score)
    if code is None:
        raise ValueError("score must be 'softmax' or 'sigmoid', got %r" % (score,))
    return code


def route(logits: torch.Tensor, k: int, *, score: str = "softmax", bias: torch.Tensor | None = None,
          groups: int = 1, groups_kept: int = 1, group_top: int = 1, renormalize: bool = True,
          scale: float = 1.0):
    """The k experts of every token and their weights (mxfp8_route).

    logits fp32 or bf16 [T, E] (rows contiguous, any row stride).  Scores are
    softmax or sigmoid of the logits; ``bias`` (fp32 [E]) is added for the
    choice only; with ``groups`` > 1 the experts form that many runs, of which
    the ``groups_kept`` with the best score stay (a run's score: its largest
    biased score, or the sum of its two largest with group_top 2).  Returns
    (ids int32 [T, k] by falling score, lowest index first among equals;
    weights fp32 [T, k]: the unbiased scores, over their sum if
    ``renormalize``, times ``scale``)."""
    code, ld = need_rows(logits, "logits")
    T, E = logits.shape
    if bias is not None:
        _need(bias, torch.float32, "bias")
        if bias.numel() != E:
            raise ValueError("bias must have E = %d entries" % E)
        same_device(logits, bias)
    sc = _score_code(score)
    ids = logits.new_empty((T, k), dtype=torch.int32)
    weights = logits.new_empty((T, k), dtype=torch.float32)
    _check(tokens_lib().mxfp8_route(_ptr(logits), code, ld, T, E, k, sc, _ptr(bias) if bias is not None else None,
                                    groups, groups_kept, group_top, renormalize, scale, _ptr(ids), _ptr(weights),
                                    _stream(logits.device)), "mxfp8_route")
    return ids, weights


def route_backward(logits: torch.Tensor, ids: torch.Tensor, d_weights: torch.Tensor, *, score: str = "softmax",
                   renormalize: bool = True, scale: float = 1.0) -> torch.Tensor:
    """Gradient of route's weights with respect to the logits, [T, E] in the
    logits' dtype (mxfp8_route_backward); arguments as route was given them."""
    code, ld = need_rows(logits, "logits")
    T, E = logits.shape
    _need(ids, torch.int32, "ids")
    _need(d_weights, torch.float32, "d_weights")
    if ids.dim() != 2 or ids.shape[0] != T or d_weights.shape != ids.shape:
        raise ValueError("ids and d_weights must both be [T = %d, k]" % T)
    same_device(logits, ids, d_weights)
    sc = _score_code(score)
    out = logits.new_empty((T, E))
    _check(tokens_lib().mxfp8_route_backward(_ptr(logits), code, ld, T, E, ids.shape[1], sc, _ptr(ids),
                                             _ptr(d_weights), renormalize, scale, _ptr(out),
                                             _stream(logits.device)), "mxfp8_route_backward")
    return out


@dataclass
class RouteTables:
    """Row tables of an expert-sorted batch (mxfp8_route_tables)."""
    offsets: torch.Tensor       # int32 [E + 1]: padded group starts, the grouped GEMMs' offsets
    counts: torch.Tensor        # int32 [E]
    row_token: torch.Tensor     # int64 [rows]: -1 for padding rows
    pair_row: torch.Tensor      # int32 [T, k]: -1 for a pair without an expert
    pad: int


def route_rows(pairs: int, experts: int, pad: int = 32) -> int:
    """Rows that ``pairs`` (token, expert) pairs over ``experts`` padded groups take at most."""
    return int(tokens_lib().mxfp8_route_rows(pairs, experts, pad))


def route_tables(ids: torch.Tensor, experts: int, pad: int = 32, rows: int | None = None) -> RouteTables:
    """Expert ids int32 [T, k] -> RouteTables: pairs sorted by (expert, token),
    groups padded to ``pad`` rows.  ``rows`` (default: route_rows, the most
    they can take) sizes row_token.  An id outside [0, experts) gets no row."""
    _need(ids, torch.int32, "ids")
    if ids.dim() != 2:
        raise ValueError("ids must be [T, k]")
    T, k = ids.shape
    L = tokens_lib()
    if rows is None:
        rows = int(L.mxfp8_route_rows(T * k, experts, pad))
    dev = ids.device
    if T == 0:
        return RouteTables(torch.zeros(experts + 1, dtype=torch.int32, device=dev),
                           torch.zeros(experts, dtype=torch.int32, device=dev),
                           torch.full((rows,), -1, dtype=torch.int64, device=dev),
                           torch.empty((0, k), dtype=torch.int32, device=dev), pad)
    offsets = ids.new_empty(experts + 1)
    counts = ids.new_empty(experts)
    row_token = ids.new_empty(rows, dtype=torch.int64)
    pair_row = torch.empty_like(ids)
    need = int(L.mxfp8_route_tables_workspace_bytes(T, k, experts))
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _check(L.mxfp8_route_tables(_ptr(ids), T, k, experts, pad, _ptr(offsets), _ptr(counts), _ptr(row_token), rows,
                                _ptr(pair_row), _ptr(ws) if need else None, need, _stream(dev)),
           "mxfp8_route_tables")
    return RouteTables(offsets, counts, row_token, pair_row, pad)


def _combine_args(y, pair_row, weights):
    _need(y, y.dtype if isinstance(y, torch.Tensor) else None, "y")
    code, _ = need_rows(y, "y")
    _need(pair_row, torch.int32, "pair_row")
    _need(weights, torch.float32, "weights")
    if pair_row.dim() != 2 or weights.shape != pair_row.shape:
        raise ValueError("pair_row and weights must both be [T, k]")
    same_device(y, pair_row, weights)
    return code


def moe_combine(y: torch.Tensor, pair_row: torch.Tensor, weights: torch.Tensor,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] * y[pair_row[t, j]] in fp32, rounded once
    to y's dtype (mxfp8_moe_combine).  y fp32 or bf16 [rows, H]."""
    code = _combine_args(y, pair_row, weights)
    T, k = pair_row.shape
    rows, H = y.shape
    if out is None:
        out = y.new_empty((T, H))
    else:
        _need(out, y.dtype, "out")
        if tuple(out.shape) != (T, H):
            raise ValueError("out must be [T, H]")
        same_device(y, out)
    _check(tokens_lib().mxfp8_moe_combine(_ptr(y), code, rows, H, _ptr(pair_row), _ptr(weights), T, k, _ptr(out),
                                          _stream(y.device)), "mxfp8_moe_combine")
    return out


def moe_combine_backward(d_out: torch.Tensor, y: torch.Tensor, pair_row: torch.Tensor, weights: torch.Tensor,
                         row_token: torch.Tensor):
    """Gradients of moe_combine: (d_y [rows, H] in y's dtype, zeros in padding
    rows; d_weights fp32 [T, k]) (mxfp8_moe_combine_backward)."""
    code = _combine_args(y, pair_row, weights)
    T, k = pair_row.shape
    rows, H = y.shape
    _need(d_out, y.dtype, "d_out")
    _need(row_token, torch.int64, "row_token")
    if tuple(d_out.shape) != (T, H) or row_token.numel() != rows:
        raise ValueError("d_out must be [T = %d, H = %d] and row_token [%d]" % (T, H, rows))
    same_device(y, d_out, row_token)
    d_y = torch.empty_like(y)
    d_w = torch.empty_like(weights)
    _check(tokens_lib().mxfp8_moe_combine_backward(_ptr(d_out), _ptr(y), code, rows, H, _ptr(pair_row),
                                                   _ptr(weights), _ptr(row_token), T, k, _ptr(d_y), _ptr(d_w),
                                                   _stream(y.device)), "mxfp8_moe_combine_backward")
    return d_y, d_w
