"""Signatures and argument checks shared by the calls of
include/mxfp8_policy.h."""
from __future__ import annotations

import ctypes

import torch

from . import lib
from ._tokens import ERR_SHAPE, need, need_rows, same_device, stream_of as _stream_of  # noqa: F401

_ready = None
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

_count = getattr(torch._C, "_increment_version", None) or torch.autograd.graph.increment_version


def stream_of(device: int) -> int:
    """The current stream of the tensors' device, which has to be the current
    one: the calls launch there, whatever device their addresses belong to."""
    if device != _current_device():
        raise ValueError("the tensors are on cuda:%d, but the current device is cuda:%d" % (device, _current_device()))
    return _stream_of(device)


def written(t: torch.Tensor) -> None:
    """The call has changed t through its address.  Autograd, which sees only
    torch's own operations, learns it from the version counter and raises its
    usual error where it still needs the former values."""
    _count((t,))


def policy_lib():
    """The library with these calls' signatures set."""
    global _ready
    if _ready is not None:
        return _ready
    L = lib()
    P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    for name, args, res in (
            ("mxfp8_swiglu", [P, I64, I64, I64, P, P, P, I32, P, P, P], I32),
            ("mxfp8_swiglu_backward", [P, I64, I64, I64, P, P, P, P, P], I32),
            ("mxfp8_lora_add_workspace_bytes", [I64] * 5, SZ),
            ("mxfp8_lora_add", [P, I32, I64, P, I64, I64, P, P, P, I64, I64, I64, I64, P, P, I64, P, P, SZ, P], I32),
            ("mxfp8_lora_backward_workspace_bytes", [I64] * 5, SZ),
            ("mxfp8_lora_backward", [P, I64, P, I64, P, P, I32, I64, I64, P, P, P, I64, I64, I64, I64, P, P, I64, P, P,
                                     P, P, SZ, P], I32),
            ("mxfp8_verify_drafts_workspace_bytes", [I64, I64, I64, I32], SZ),
            ("mxfp8_verify_drafts", [P, I32, I64, I64, I64, P, I64, P, P, P, I64, P, I64, ctypes.c_double, P, P, P, P, SZ,
                                     P], I32)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res
    _ready = L
    return L


def need_bf16_rows(t, name: str) -> int:
    """The row stride of a 2-D bf16 device tensor whose rows are contiguous."""
    code, ld = need_rows(t, name)
    if t.dtype is not torch.bfloat16:
        raise TypeError("%s must be torch.bfloat16, got %s" % (name, t.dtype))
    return ld
