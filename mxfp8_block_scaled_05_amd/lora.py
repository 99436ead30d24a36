"""Low-rank adapters of many requests beside a shared projection
(include/mxfp8_policy.h).

    t      = route_tables(adapter_ids.view(-1, 1), E)      # once for all the layers of a batch
    y      = gemm_packed(x_grid, w, torch.bfloat16)         # the shared projection
    hidden = lora_add_(y, x, a, b, t, scales, keep_hidden=True)
    d_a, d_b = lora_backward_(d_x, d_y, x_grid, a, b, hidden, t, scales)
"""
from __future__ import annotations

import torch

from . import PackedWeight, _check, packed_bytes
from ._policy import ERR_SHAPE, need, need_bf16_rows, need_rows, policy_lib, same_device, stream_of, written

_BF16, _CANONICAL, _PACKED = 0, 1, 2


def _adapters(a, b, scales, tables):
    """(E, r, K, N, pointers of a, b, scales, offsets, row_token, rows)"""
    pa, pb = need(a, torch.bfloat16, "a"), need(b, torch.bfloat16, "b")
    if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
        raise ValueError("a must be [E, r, K] and b [E, N, r], got %s and %s" % (tuple(a.shape), tuple(b.shape)))
    E, r, K = a.shape
    ps = None
    if scales is not None:
        ps = need(scales, torch.float32, "scales")
        if scales.numel() != E:
            raise ValueError("scales must have E = %d entries" % E)
    po, pr = need(tables.offsets, torch.int32, "tables.offsets"), need(tables.row_token, torch.int64, "tables.row_token")
    rows = tables.row_token.numel()
    if tables.offsets.numel() != E + 1 or tables.pad % 32 or rows % 32:
        raise ValueError("tables must be of E = %d adapters, padded to a multiple of 32 rows" % E)
    return E, r, K, b.shape[1], pa, pb, ps, po, pr, rows


def lora_add_(y: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, tables,
              scales: torch.Tensor | None = None, *, keep_hidden: bool = False) -> torch.Tensor | None:
    """y[t] += scales[e] * b[e] @ (a[e] @ x[t]) in place, e the adapter of row t
    (mxfp8_lora_add).  y fp32 or bf16 [T, N], x bf16 [T, K] (rows contiguous,
    strides of whole 16 bytes), a bf16 [E, r, K], b bf16 [E, N, r], scales fp32
    [E] or None (all 1); ``tables`` = route_tables(ids int32 [T, 1], E): rows
    with an id outside [0, E) stay as they are.  Returns the hidden rows, fp32
    [rows, r] in the tables' order, for lora_backward_ with ``keep_hidden``."""
    E, r, K, N, pa, pb, ps, po, pr, rows = _adapters(a, b, scales, tables)
    code, ld_y = need_rows(y, "y")
    ld_x = need_bf16_rows(x, "x")
    T = x.shape[0]
    if x.shape[1] != K or tuple(y.shape) != (T, N):
        raise ValueError("x must be [T, K = %d] and y [T, N = %d], got %s and %s" % (K, N, tuple(x.shape), tuple(y.shape)))
    dev = same_device(y, x, a, b, scales, tables.offsets, tables.row_token)
    L = policy_lib()
    need_ws = L.mxfp8_lora_add_workspace_bytes(rows, E, r, K, N)
    if not need_ws and rows:
        _check(ERR_SHAPE, "mxfp8_lora_add")
    ws = a.new_empty(need_ws // 2)
    hidden = ws.new_empty((rows, r), dtype=torch.float32) if keep_hidden else None
    _check(L.mxfp8_lora_add(y.data_ptr(), code, ld_y, x.data_ptr(), ld_x, T, pa, pb, ps, E, r, K, N, po, pr, rows,
                            hidden.data_ptr() if keep_hidden else None, ws.data_ptr(), need_ws, stream_of(dev)),
           "mxfp8_lora_add")
    written(y)
    return hidden


def _input(x, T, K):
    """(form, pointer, scales' pointer, row stride, tensors) of the adapters' input"""
    if isinstance(x, PackedWeight):
        if (x.batch, x.N, x.K) != (1, T, K):
            raise ValueError("x must be PackedWeight(batch 1, N = %d, K = %d)" % (T, K))
        q, s = need(x.q, torch.uint8, "x.q"), need(x.s, torch.uint8, "x.s")
        if x.q.numel() < packed_bytes(1, T, K, 0) or x.s.numel() < packed_bytes(1, T, K, 1):
            raise ValueError("x's buffers are too small")
        return _PACKED, q, s, K, (x.q, x.s)
    if isinstance(x, (tuple, list)):
        q, s = need(x[0], torch.uint8, "x's codes"), need(x[1], torch.uint8, "x's scales")
        if tuple(x[0].shape) != (T, K) or tuple(x[1].shape) != (T, K // 32):
            raise ValueError("x must be codes [T = %d, K = %d] and scales [T, K / 32]" % (T, K))
        return _CANONICAL, q, s, K, tuple(x)
    ld = need_bf16_rows(x, "x")
    if tuple(x.shape) != (T, K):
        raise ValueError("x must be [T = %d, K = %d]" % (T, K))
    return _BF16, x.data_ptr(), None, ld, (x,)


def lora_backward_(d_x: torch.Tensor | None, d_y: torch.Tensor, x, a: torch.Tensor, b: torch.Tensor,
                   hidden: torch.Tensor, tables, scales: torch.Tensor | None = None):
    """Gradients of lora_add_ (mxfp8_lora_backward): adds the adapters' share to
    d_x (bf16 [T, K], what the shared projection's own product gave; None: left
    out) and returns (d_a fp32 [E, r, K], d_b fp32 [E, N, r]).  d_y bf16 [T, N].
    ``x`` is the input in bf16 [T, K], or kept in 8 bits: (q, s) as quantize(x,
    1) gives it, or the PackedWeight that the shared projection read."""
    E, r, K, N, pa, pb, ps, po, pr, rows = _adapters(a, b, scales, tables)
    ld_dy = need_bf16_rows(d_y, "d_y")
    T = d_y.shape[0]
    if d_y.shape[1] != N:
        raise ValueError("d_y must be [T, N = %d]" % N)
    form, px, pxs, ld_x, xs = _input(x, T, K)
    ld_dx = K
    if d_x is not None:
        ld_dx = need_bf16_rows(d_x, "d_x")
        if tuple(d_x.shape) != (T, K):
            raise ValueError("d_x must be [T = %d, K = %d]" % (T, K))
    ph = need(hidden, torch.float32, "hidden")
    if tuple(hidden.shape) != (rows, r):
        raise ValueError("hidden must be [rows = %d, r = %d]" % (rows, r))
    dev = same_device(d_y, d_x, *xs, a, b, scales, hidden, tables.offsets, tables.row_token)
    L = policy_lib()
    need_ws = L.mxfp8_lora_backward_workspace_bytes(rows, E, r, K, N)
    if not need_ws:
        _check(ERR_SHAPE, "mxfp8_lora_backward")
    ws = a.new_empty(need_ws // 2)
    d_a = hidden.new_empty(E, r, K)
    d_b = hidden.new_empty(E, N, r)
    _check(L.mxfp8_lora_backward(d_x.data_ptr() if d_x is not None else None, ld_dx, d_y.data_ptr(), ld_dy, px, pxs, form,
                                 ld_x, T, pa, pb, ps, E, r, K, N, po, pr, rows, ph, d_a.data_ptr(), d_b.data_ptr(),
                                 ws.data_ptr(), need_ws, stream_of(dev)), "mxfp8_lora_backward")
    if d_x is not None:
        written(d_x)
    return d_a, d_b
