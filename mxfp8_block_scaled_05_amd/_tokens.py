"""Signatures and argument checks shared by the token-level operators
(include/mxfp8_tokens.h)."""
from __future__ import annotations

import ctypes

import torch

from . import MXFP8_BF16, MXFP8_F32, _need, _raw_stream as stream_of, lib  # noqa: F401

_ready = None


def tokens_lib():
    """The library with the token-level calls' signatures set."""
    global _ready
    if _ready is not None:
        return _ready
    L = lib()
    P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    F, D = ctypes.c_float, ctypes.c_double
    SZ = ctypes.c_size_t
    for name, args, res in (
            ("mxfp8_route", [P, I32, I64, I64, I64, I64, I32, P, I64, I64, I64, I32, F, P, P, P], I32),
            ("mxfp8_route_backward", [P, I32, I64, I64, I64, I64, I32, P, P, I32, F, P, P], I32),
            ("mxfp8_route_rows", [I64, I64, I64], I64),
            ("mxfp8_route_tables_workspace_bytes", [I64, I64, I64], SZ),
            ("mxfp8_route_tables", [P, I64, I64, I64, I64, P, P, P, I64, P, P, SZ, P], I32),
            ("mxfp8_moe_combine", [P, I32, I64, I64, P, P, I64, I64, P, P], I32),
            ("mxfp8_moe_combine_backward", [P, P, I32, I64, I64, P, P, P, I64, I64, P, P, P], I32),
            ("mxfp8_token_logprobs_workspace_bytes", [I64, I64, I64], SZ),
            ("mxfp8_token_logprobs", [P, I32, I64, I64, I64, P, D, I64, P, P, P, P, P, P, SZ, P], I32),
            ("mxfp8_token_logprobs_backward", [P, I32, I64, I64, I64, P, P, P, P, P, D, P, I64, P], I32)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res
    _ready = L
    return L


# limits of include/mxfp8_tokens.h that have to hold before outputs are allocated
MAX_K, MAX_EXPERTS, MAX_PAD, MAX_TOP = 32, 1024, 1024, 64
ERR_SHAPE = 2

_CODES = {torch.float32: MXFP8_F32, torch.bfloat16: MXFP8_BF16}

# The checks below look at the usual tensor first and leave what is not one to
# the slower code that names the fault: a small call spends more time in
# Python than on the device.


def need(t, dtype, name: str) -> int:
    """The address of a contiguous device tensor of that dtype."""
    if t.__class__ is not torch.Tensor or t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
        _need(t, dtype, name)
    return t.data_ptr()


def need_rows(t, name: str):
    """(dtype code, row stride) of a 2-D fp32 or bf16 device tensor whose rows
    are contiguous; the rows themselves may lie further apart."""
    if t.__class__ is torch.Tensor and t.is_cuda and t.dim() == 2 and t.is_contiguous():
        code = _CODES.get(t.dtype)
        if code is not None:
            return code, t.shape[1] or 1
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError("%s must be torch.float32 or torch.bfloat16, got %s" % (name, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    rows, cols = t.shape
    ld, one = t.stride()
    if rows <= 1:
        ld = max(ld, cols, 1)
    if (one != 1 and cols > 1) or ld < cols:
        raise ValueError("the rows of %s must be contiguous and must not overlap" % name)
    return code, ld


def same_device(first, *others) -> int:
    """The index of the one device of the tensors (None: left out)."""
    d = first.get_device()
    for t in others:
        if t is not None and t.get_device() != d:
            raise ValueError("all tensors must be on one device, got %s and %s" % (first.device, t.device))
    return d
