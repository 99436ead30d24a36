"""The gradient of one row in place: a single row has no stride, whatever its
views say."""
import ctypes
import os

import pytest
import torch

import mxfp8_block_scaled_05_amd as m


def test_one_row_in_place_with_other_strides():
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libmxfp8.so not built")
    if torch.cuda.is_available():
        pytest.skip("passes pointers to host memory")
    from mxfp8_block_scaled_05_amd._tokens import tokens_lib
    buf = ctypes.create_string_buffer(8192)
    p = ctypes.c_void_p((ctypes.addressof(buf) + 15) & ~15)
    o = ctypes.c_void_p(p.value + 4096)
    call = lambda T, ld, ldo: tokens_lib().mxfp8_token_logprobs_backward(p, 0, ld, T, 100, o, o, o, o, o, 1.0, p, ldo, None)
    assert call(1, 400, 100) == call(1, 100, 100) and call(1, 100, 100) not in (0, 1, 2, 5, 8)
    assert call(2, 400, 100) == 2                               # two rows: not in place


@pytest.mark.gpu
def test_one_row_in_place(mx):
    store = torch.randn((3, 400), device="cuda")
    t, one = torch.tensor([5], device="cuda"), torch.ones(1, device="cuda")
    x = store[:1, :150]
    r = mx.token_logprobs(x, t)
    d = mx.token_logprobs_backward(x, t, r.stats, r.entropy, one, one)
    rest = store[:, 150:].clone()
    mx.token_logprobs_backward(x, t, r.stats, r.entropy, one, one, out=store[0, :150].view(1, 150))
    assert torch.equal(store[:1, :150], d) and torch.equal(store[:, 150:], rest)
