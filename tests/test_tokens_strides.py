"""Row strides of the token-level calls: any that addresses memory passes the
host checks (the call then ends at the missing GPU, or enqueues nothing)."""
import ctypes
import os

import pytest
import torch

import mxfp8_block_scaled_05_amd as m

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="passes pointers to host memory")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libmxfp8.so not built")
    from mxfp8_block_scaled_05_amd._tokens import tokens_lib
    return tokens_lib()


def _calls(L, ld):
    buf = ctypes.create_string_buffer(4096)
    p = ctypes.c_void_p((ctypes.addressof(buf) + 15) & ~15)
    o, o2, o3 = (ctypes.c_void_p(p.value + n) for n in (2048, 2560, 3072))
    yield L.mxfp8_route(p, 1, ld, 2, 64, 4, 0, None, 1, 1, 1, 1, 1.0, o, o2, None)
    yield L.mxfp8_route_backward(p, 1, ld, 2, 64, 4, 0, p, p, 1, 1.0, o, None)
    yield L.mxfp8_token_logprobs(p, 1, ld, 2, 64, p, 1.0, 0, o, o2, o3, None, None, None, 0, None)
    yield L.mxfp8_token_logprobs_backward(p, 1, ld, 2, 64, p, p, p, p, p, 1.0, o, 64, None)
    yield L.mxfp8_token_logprobs_backward(p, 1, 64, 2, 64, p, p, p, p, p, 1.0, o, ld, None)


@pytest.mark.parametrize("ld", [1 << 31, (1 << 31) + 1, 1 << 40, 1 << 59])
def test_far_rows_are_taken(L, ld):
    assert list(_calls(L, ld)) == list(_calls(L, 64))


@pytest.mark.parametrize("ld", [63, -64, (1 << 59) + 1, (1 << 63) - 1])
def test_strides_that_address_nothing(L, ld):
    assert list(_calls(L, ld)) == [2] * 5
