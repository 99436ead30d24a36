"""The gated activation with its inputs kept in 8 bits for the backward pass
(include/mxfp8_policy.h).

    r = swiglu(gu)                                   # Swiglu: h bf16, saved_q, saved_s
    r = swiglu(gu, layout="packed")                  # h as the next projection's operand
    d_gu, h = swiglu_backward(d_h, r.saved_q, r.saved_s)
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import MXFP8_CANONICAL, MXFP8_PACKED, PackedWeight, _check, packed_bytes
from ._policy import ERR_SHAPE, need, need_bf16_rows, policy_lib, same_device, stream_of


@dataclass
class Swiglu:
    h: object                               # bf16 [T, I], (q [T, I], s [T, I/32]) or PackedWeight(1, T, I)
    saved_q: torch.Tensor | None            # uint8 [T, 2 I]: E4M3 codes of gate | up
    saved_s: torch.Tensor | None            # uint8 [T, 2 I / 32]: their scales


def swiglu(gu: torch.Tensor, *, layout: str = "bf16", save: bool = True) -> Swiglu:
    """silu(gate) * up of gu = gate | up, bf16 [T, 2 I] (I % 32 == 0, rows
    contiguous, any row stride of whole 16 bytes), and with ``save`` the 8-bit
    checkpoint of gu for swiglu_backward: exactly quantize(gu, 1)
    (mxfp8_swiglu).

    ``layout`` says how h comes: "bf16" [T, I]; "canonical", the (q, s) that
    quantize(h, 1) gives; "packed", the same as the GEMMs' packed operand (T at
    least 1)."""
    ld = need_bf16_rows(gu, "gu")
    T, cols = gu.shape
    inner = cols // 2
    if cols != 2 * inner or inner % 32 or not inner:
        raise ValueError("gu must be [T, 2 I] with I a multiple of 32, got %s" % (tuple(gu.shape),))
    h = hq = hs = None
    code = MXFP8_CANONICAL
    if layout == "bf16":
        out = h = gu.new_empty(T, inner)
    elif layout == "canonical":
        hq = gu.new_empty((T, inner), dtype=torch.uint8)
        hs = hq.new_empty(T, inner // 32)
        out = (hq, hs)
    elif layout == "packed":
        if packed_bytes(1, T, inner, 0) == 0:
            _check(ERR_SHAPE, "mxfp8_swiglu")
        code = MXFP8_PACKED
        hq = gu.new_empty(packed_bytes(1, T, inner, 0), dtype=torch.uint8)
        hs = hq.new_empty(packed_bytes(1, T, inner, 1))
        out = PackedWeight(hq, hs, 1, T, inner)
    else:
        raise ValueError("layout must be 'bf16', 'canonical' or 'packed', got %r" % (layout,))
    q = s = None
    if save:
        q = gu.new_empty((T, cols), dtype=torch.uint8)
        s = q.new_empty(T, cols // 32)
    _check(policy_lib().mxfp8_swiglu(gu.data_ptr(), ld, T, inner, h.data_ptr() if hq is None else None,
                                     None if hq is None else hq.data_ptr(), None if hs is None else hs.data_ptr(), code,
                                     q.data_ptr() if save else None, s.data_ptr() if save else None,
                                     stream_of(gu.get_device())), "mxfp8_swiglu")
    return Swiglu(out, q, s)


def swiglu_backward(d_h: torch.Tensor, saved_q: torch.Tensor, saved_s: torch.Tensor, *, recompute: bool = True):
    """(d_gu bf16 [T, 2 I], h bf16 [T, I] or None) from the gradient of h (bf16
    [T, I], rows contiguous) and swiglu's checkpoint: the gradient at the
    checkpoint's values, and with ``recompute`` the product of those values
    again, for the next projection's weight gradient (mxfp8_swiglu_backward)."""
    ld = need_bf16_rows(d_h, "d_h")
    q, s = need(saved_q, torch.uint8, "saved_q"), need(saved_s, torch.uint8, "saved_s")
    T, inner = d_h.shape
    if tuple(saved_q.shape) != (T, 2 * inner) or tuple(saved_s.shape) != (T, inner // 16):
        raise ValueError("saved_q and saved_s must be [T = %d, 2 I = %d] and [T, 2 I / 32], got %s and %s"
                         % (T, 2 * inner, tuple(saved_q.shape), tuple(saved_s.shape)))
    dev = same_device(d_h, saved_q, saved_s)
    d_gu = d_h.new_empty(T, 2 * inner)
    h = d_h.new_empty(T, inner) if recompute else None
    _check(policy_lib().mxfp8_swiglu_backward(d_h.data_ptr(), ld, T, inner, q, s, d_gu.data_ptr(),
                                              h.data_ptr() if recompute else None, stream_of(dev)),
           "mxfp8_swiglu_backward")
    return d_gu, h
