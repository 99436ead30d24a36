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

from . import _check
from ._tokens import ERR_SHAPE, MAX_EXPERTS, MAX_K, MAX_PAD, need, need_rows, same_device, stream_of, tokens_lib

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
    b = None
    if bias is not None:
        b = need(bias, torch.float32, "bias")
        if bias.numel() != E:
            raise ValueError("bias must have E = %d entries" % E)
    dev = same_device(logits, bias)
    sc = _score_code(score)
    if not 0 < k <= MAX_K:
        _check(ERR_SHAPE, "mxfp8_route")
    ids = logits.new_empty((T, k), dtype=torch.int32)
    weights = torch.empty_like(ids, dtype=torch.float32)
    _check(tokens_lib().mxfp8_route(logits.data_ptr(), code, ld, T, E, k, sc, b, groups, groups_kept, group_top,
                                    renormalize, scale, ids.data_ptr(), weights.data_ptr(), stream_of(dev)),
           "mxfp8_route")
    return ids, weights


def route_backward(logits: torch.Tensor, ids: torch.Tensor, d_weights: torch.Tensor, *, score: str = "softmax",
                   renormalize: bool = True, scale: float = 1.0) -> torch.Tensor:
    """Gradient of route's weights with respect to the logits, [T, E] in the
    logits' dtype (mxfp8_route_backward); arguments as route was given them."""
    code, ld = need_rows(logits, "logits")
    T, E = logits.shape
    i, d = need(ids, torch.int32, "ids"), need(d_weights, torch.float32, "d_weights")
    if ids.dim() != 2 or ids.shape[0] != T or d_weights.shape != ids.shape:
        raise ValueError("ids and d_weights must both be [T = %d, k]" % T)
    dev = same_device(logits, ids, d_weights)
    sc = _score_code(score)
    out = logits.new_empty(T, E)
    _check(tokens_lib().mxfp8_route_backward(logits.data_ptr(), code, ld, T, E, ids.shape[1], sc, i, d, renormalize,
                                             scale, out.data_ptr(), stream_of(dev)), "mxfp8_route_backward")
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
    i = need(ids, torch.int32, "ids")
    if ids.dim() != 2:
        raise ValueError("ids must be [T, k]")
    T, k = ids.shape
    L = tokens_lib()
    if not 0 < experts <= MAX_EXPERTS or not 0 < pad <= MAX_PAD or (rows is not None and not 0 <= rows < 1 << 31):
        _check(ERR_SHAPE, "mxfp8_route_tables")
    if rows is None:
        rows = int(L.mxfp8_route_rows(T * k, experts, pad))
    if T == 0:
        dev = ids.device
        return RouteTables(torch.zeros(experts + 1, dtype=torch.int32, device=dev),
                           torch.zeros(experts, dtype=torch.int32, device=dev),
                           torch.full((rows,), -1, dtype=torch.int64, device=dev),
                           torch.empty((0, k), dtype=torch.int32, device=dev), pad)
    offsets = ids.new_empty(experts + 1)
    counts = ids.new_empty(experts)
    row_token = ids.new_empty(rows, dtype=torch.int64)
    pair_row = torch.empty_like(ids)
    need_ws = L.mxfp8_route_tables_workspace_bytes(T, k, experts)
    ws = ids.new_empty(need_ws // 4) if need_ws else None
    _check(L.mxfp8_route_tables(i, T, k, experts, pad, offsets.data_ptr(), counts.data_ptr(), row_token.data_ptr(), rows,
                                pair_row.data_ptr(), ws.data_ptr() if need_ws else None, need_ws,
                                stream_of(ids.get_device())), "mxfp8_route_tables")
    return RouteTables(offsets, counts, row_token, pair_row, pad)


def _combine_args(y, pair_row, weights):
    code, _ = need_rows(y, "y")
    if not y.is_contiguous():
        raise ValueError("y must be contiguous")
    p, w = need(pair_row, torch.int32, "pair_row"), need(weights, torch.float32, "weights")
    if pair_row.dim() != 2 or weights.shape != pair_row.shape:
        raise ValueError("pair_row and weights must both be [T, k]")
    return code, p, w


def moe_combine(y: torch.Tensor, pair_row: torch.Tensor, weights: torch.Tensor,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] * y[pair_row[t, j]] in fp32, rounded once
    to y's dtype (mxfp8_moe_combine).  y fp32 or bf16 [rows, H]; ``out`` must not
    share memory with it."""
    code, p, w = _combine_args(y, pair_row, weights)
    T, k = pair_row.shape
    rows, H = y.shape
    if out is None:
        out = y.new_empty(T, H)
    else:
        need(out, y.dtype, "out")
        if tuple(out.shape) != (T, H):
            raise ValueError("out must be [T, H]")
    dev = same_device(y, pair_row, weights, out)
    _check(tokens_lib().mxfp8_moe_combine(y.data_ptr(), code, rows, H, p, w, T, k, out.data_ptr(), stream_of(dev)),
           "mxfp8_moe_combine")
    return out


def moe_combine_backward(d_out: torch.Tensor, y: torch.Tensor, pair_row: torch.Tensor, weights: torch.Tensor,
                         row_token: torch.Tensor):
    """Gradients of moe_combine: (d_y [rows, H] in y's dtype, zeros in padding
    rows; d_weights fp32 [T, k]) (mxfp8_moe_combine_backward)."""
    code, p, w = _combine_args(y, pair_row, weights)
    T, k = pair_row.shape
    rows, H = y.shape
    d, r = need(d_out, y.dtype, "d_out"), need(row_token, torch.int64, "row_token")
    if tuple(d_out.shape) != (T, H) or row_token.numel() != rows:
        raise ValueError("d_out must be [T = %d, H = %d] and row_token [%d]" % (T, H, rows))
    dev = same_device(y, pair_row, weights, d_out, row_token)
    d_y = torch.empty_like(y)
    d_w = torch.empty_like(weights)
    _check(tokens_lib().mxfp8_moe_combine_backward(d, y.data_ptr(), code, rows, H, p, w, r, T, k, d_y.data_ptr(),
                                                   d_w.data_ptr(), stream_of(dev)), "mxfp8_moe_combine_backward")
    return d_y, d_w
