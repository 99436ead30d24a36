"""An output of a token-level call that shares memory with another buffer of the
call is refused on the host; buffers beside and between each other are not."""
import ctypes
import os
import random

import pytest
import torch

import mxfp8_block_scaled_05_amd as m

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="passes pointers to host memory")

OVERLAP = 8


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libmxfp8.so not built")
    from mxfp8_block_scaled_05_amd._tokens import tokens_lib
    return tokens_lib()


class Space:
    """Addresses in host memory, never read: each buffer of a call 2^20 bytes from the next."""

    def __init__(self):
        self.store = ctypes.create_string_buffer(16 << 20)
        self.base = (ctypes.addressof(self.store) + 63) & ~63

    def __getitem__(self, slot):
        return ctypes.c_void_p(self.base + (slot << 20))


def _check(call, sizes, outputs, allowed=()):
    """call(addresses) with buffers of those sizes: apart it gets past the host checks, and any output moved onto the
    first or the last byte of another buffer is refused (the pairs in `allowed` may be one buffer)."""
    space = Space()
    apart = [space[i] for i in range(len(sizes))]
    fine = call(*apart)
    assert fine not in (0, 1, 2, 3, 4, 5, OVERLAP)                          # no GPU here: that is all it misses
    for o in outputs:
        for i in range(len(sizes)):
            if i == o:
                continue
            for at, want in ((0, OVERLAP), (-sizes[o] + 8, OVERLAP), (sizes[i] - 8, OVERLAP), (-sizes[o], fine), (sizes[i], fine)):
                if at == 0 and (o, i) in allowed:
                    want = fine
                moved = list(apart)
                moved[o] = ctypes.c_void_p(apart[i].value + at)
                assert call(*moved) == want, (o, i, at)


def test_route(L):
    _check(lambda x, ids, w, b: L.mxfp8_route(x, 0, 64, 6, 64, 4, 0, b, 1, 1, 1, 1, 1.0, ids, w, None),
           (6 * 256, 96, 96, 256), (1, 2))
    _check(lambda x, ids, w: L.mxfp8_route(x, 1, 64, 6, 64, 4, 0, None, 1, 1, 1, 1, 1.0, ids, w, None), (6 * 128, 96, 96), (1, 2))


def test_route_backward(L):
    _check(lambda x, ids, dw, dx: L.mxfp8_route_backward(x, 0, 64, 6, 64, 4, 0, ids, dw, 1, 1.0, dx, None),
           (6 * 256, 96, 96, 6 * 256), (3,))


def test_route_tables(L):
    rows = L.mxfp8_route_rows(128, 8, 32)
    _check(lambda ids, off, cnt, tok, pr: L.mxfp8_route_tables(ids, 32, 4, 7, 32, off, cnt, tok, rows, pr, None, 0, None),
           (512, 32, 28 + 4, rows * 8, 512), (1, 3, 4))
    rows = L.mxfp8_route_rows(1 << 15, 8, 32)
    ws = L.mxfp8_route_tables_workspace_bytes(1 << 13, 4, 8)
    assert ws > 0
    _check(lambda ids, off, cnt, tok, pr, w: L.mxfp8_route_tables(ids, 1 << 13, 4, 8, 32, off, cnt, tok, rows, pr, w, ws, None),
           (1 << 17, 40, 32, rows * 8, 1 << 17, ws), (2, 4, 5))


def test_combine(L):
    _check(lambda y, pr, w, out: L.mxfp8_moe_combine(y, 1, 64, 100, pr, w, 8, 2, out, None), (64 * 200, 64, 64, 8 * 200), (3,))


def test_combine_backward(L):
    _check(lambda d, y, pr, w, tok, dy, dw: L.mxfp8_moe_combine_backward(d, y, 0, 64, 100, pr, w, tok, 8, 2, dy, dw, None),
           (8 * 400, 64 * 400, 64, 64, 512, 64 * 400, 64), (5, 6), allowed=((5, 1), (6, 3)))


def test_logprobs(L):
    _check(lambda x, t, lp, H, st, tl, ti: L.mxfp8_token_logprobs(x, 0, 100, 6, 100, t, 1.0, 4, lp, H, st, tl, ti, None, 0, None),
           (2400, 48, 24, 24, 48, 96, 192), (2, 3, 4, 5, 6))
    need = L.mxfp8_token_logprobs_workspace_bytes(2, 20000, 0)
    assert need > 0 and need % 16 == 0
    space = Space()
    call = lambda ws, n: L.mxfp8_token_logprobs(space[0], 1, 20000, 2, 20000, space[1], 1.0, 0, space[2], space[3], space[4], None, None,
                                                ws, n, None)
    fine = call(space[5], need)
    inside = ctypes.c_void_p(space[0].value + 64)
    assert call(inside, need) == OVERLAP and call(inside, need - 1) == fine and fine not in (0, 1, 2, 5)


def test_logprobs_backward(L):
    _check(lambda x, t, st, H, g, h, dx: L.mxfp8_token_logprobs_backward(x, 0, 100, 6, 100, t, st, H, g, h, 1.0, dx, 100, None),
           (2400, 48, 48, 24, 24, 24, 2400), (6,), allowed=((6, 0),))


def test_strided_rows(L):
    """Rows of the logits and of their gradient, anywhere in one buffer, against the bytes themselves."""
    space = Space()
    rest = [space[i] for i in range(8, 13)]
    fine = L.mxfp8_token_logprobs_backward(space[0], 1, 10, 3, 10, *rest, 1.0, space[4], 10, None)
    assert fine not in (0, 1, 2, 4, 5, OVERLAP)
    rng = random.Random(5)
    seen = set()
    for _ in range(6000):
        T, V = rng.randint(1, 7), rng.randint(1, 12)
        ld, ldo = V + rng.choice([0, 1, 5, V, 40]), V + rng.choice([0, 1, 3, V, 17, 40])
        if rng.random() < 0.4:
            ldo = ld
        at = rng.randint(-T * ldo - 3, T * ld + 3)
        if at == 0 and ld != ldo:
            continue                                                        # refused as a size
        a = {i * ld + c for i in range(T) for c in range(V)}
        b = {at + i * ldo + c for i in range(T) for c in range(V)}
        want = OVERLAP if a & b and at != 0 else fine
        x = ctypes.c_void_p(space[2].value)
        got = L.mxfp8_token_logprobs_backward(x, 1, ld, T, V, *rest, 1.0, ctypes.c_void_p(x.value + 2 * at), ldo, None)
        assert got == want, (T, V, ld, ldo, at)
        seen.add((bool(a & b), ld == ldo, T > 1))
    assert len(seen) == 8
