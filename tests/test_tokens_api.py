"""Token-level operators without a GPU: the C entry points refuse bad
arguments on the host before any device work, the host-only size functions,
and the Python calls' own checks."""
import ctypes
import os
import re

import pytest
import torch

import mxfp8_block_scaled_05_amd as m

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL = None


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libmxfp8.so not built")
    from mxfp8_block_scaled_05_amd._tokens import tokens_lib
    return tokens_lib()


@pytest.fixture(scope="module")
def p():
    buf = ctypes.create_string_buffer(4096 + 16)
    ptr = ctypes.c_void_p((ctypes.addressof(buf) + 15) & ~15)
    ptr._keep = buf
    return ptr


def _off(p, n):
    return ctypes.c_void_p(p.value + n)


def test_library_exports_every_declared_symbol(L):
    src = open(os.path.join(ROOT, "include", "mxfp8_tokens.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(mxfp8_[a-z_0-9]+)\s*\(", src)))
    assert len(names) == 10
    for n in names:
        assert hasattr(L, n), n


def _route(L, p, x=0, dtype=0, ld=64, T=4, E=64, k=4, score=0, bias=NULL, groups=1, kept=1, gtop=1, ids=0, w=0):
    pick = lambda v: p if v == 0 else v
    return L.mxfp8_route(pick(x), dtype, ld, T, E, k, score, bias, groups, kept, gtop, 1, 1.0, pick(ids), pick(w), NULL)


def test_route_refusals(L, p):
    r = lambda **a: _route(L, p, **a)
    assert r(x=NULL) == 1 and r(ids=NULL) == 1 and r(w=NULL) == 1
    assert r(dtype=2) == 4 and r(score=2) == 4
    for bad in (dict(T=-1), dict(T=1 << 26), dict(E=0), dict(E=513, ld=513), dict(k=0), dict(k=33), dict(k=65),
                dict(ld=63), dict(groups=0), dict(groups=3, kept=1), dict(groups=4, kept=0), dict(groups=4, kept=5),
                dict(groups=4, kept=1, gtop=0), dict(groups=4, kept=1, gtop=3), dict(groups=64, kept=64, gtop=2),
                dict(groups=32, kept=1, k=4), dict(E=8, ld=8, k=9)):
        assert r(**bad) == 2, bad
    assert r(x=_off(p, 2)) == 5 and r(x=_off(p, 1), dtype=1) == 5
    assert r(bias=_off(p, 1)) == 5 and r(ids=_off(p, 2)) == 5 and r(w=_off(p, 2)) == 5
    assert r(T=0, x=NULL, ids=NULL, w=NULL) == 0                        # no tokens: nothing to do


def test_route_backward_refusals(L, p):
    def r(x=p, dtype=0, ld=64, T=4, E=64, k=4, score=0, ids=p, dw=p, dx=p):
        return L.mxfp8_route_backward(x, dtype, ld, T, E, k, score, ids, dw, 1, 1.0, dx, NULL)
    for n in ("x", "ids", "dw", "dx"):
        assert r(**{n: NULL}) == 1, n
        assert r(**{n: _off(p, 1)}) == 5, n
    assert r(dtype=5) == 4 and r(score=-1) == 4
    for bad in (dict(T=-1), dict(E=0), dict(E=513, ld=513), dict(k=33), dict(k=0), dict(ld=10)):
        assert r(**bad) == 2, bad
    assert r(T=0, x=NULL) == 0


def test_route_rows(L):
    for pairs, E, pad in ((0, 4, 32), (1, 4, 32), (5, 4, 32), (256, 128, 32), (1000, 3, 1), (7, 1024, 1024),
                          (131072, 256, 128)):
        # the most a placement can take: every used expert one row over a multiple of pad
        used = min(E, pairs)
        most = 0
        for u in range(max(0, used - 3), used + 1):
            if u == 0:
                continue
            extra = (pairs - u) // pad                 # u groups of one row, the rest in whole multiples
            most = max(most, (u + extra) * pad)
        got = L.mxfp8_route_rows(pairs, E, pad)
        assert got % pad == 0 and most <= got <= pairs + used * (pad - 1), (pairs, E, pad)
    for bad in ((-1, 4, 32), (4, 0, 32), (4, 1025, 32), (4, 4, 0), (4, 4, 1025), (1 << 31, 4, 32)):
        assert L.mxfp8_route_rows(*bad) == 0


def test_route_tables_refusals(L, p):
    rows = L.mxfp8_route_rows(16, 8, 32)

    def r(ids=p, T=4, k=4, E=8, pad=32, off=p, cnt=p, tok=p, rows=rows, pr=p, ws=NULL, nws=0):
        return L.mxfp8_route_tables(ids, T, k, E, pad, off, cnt, tok, rows, pr, ws, nws, NULL)
    for n in ("ids", "off", "cnt", "tok", "pr"):
        assert r(**{n: NULL}) == 1, n
        assert r(**{n: _off(p, 1)}) == 5, n
    assert r(tok=_off(p, 4)) == 5                                       # int64
    for bad in (dict(T=0), dict(k=0), dict(E=0), dict(E=1025), dict(pad=0), dict(pad=1025), dict(rows=rows - 1),
                dict(rows=1 << 31), dict(T=1 << 30, k=4)):
        assert r(**bad) == 2, bad
    need = L.mxfp8_route_tables_workspace_bytes(4096, 8, 8)
    big = dict(T=4096, k=8, rows=1 << 20)
    assert need > 0 and r(ws=NULL, nws=need, **big) == 1
    assert r(ws=p, nws=need - 1, **big) == 2 and r(ws=_off(p, 2), nws=need, **big) == 5
    assert L.mxfp8_route_tables_workspace_bytes(32, 8, 128) == 0
    assert L.mxfp8_route_tables_workspace_bytes(0, 8, 128) == 0


def test_combine_refusals(L, p):
    def f(y=p, dtype=1, rows=64, H=64, pr=p, w=p, T=4, k=2, out=p):
        return L.mxfp8_moe_combine(y, dtype, rows, H, pr, w, T, k, out, NULL)

    def b(d=p, y=p, dtype=1, rows=64, H=64, pr=p, w=p, tok=p, T=4, k=2, dy=p, dw=p):
        return L.mxfp8_moe_combine_backward(d, y, dtype, rows, H, pr, w, tok, T, k, dy, dw, NULL)
    for n in ("y", "pr", "w", "out"):
        assert f(**{n: NULL}) == 1 and f(**{n: _off(p, 1)}) == 5, n
    for n in ("d", "y", "pr", "w", "tok", "dy", "dw"):
        assert b(**{n: NULL}) == 1 and b(**{n: _off(p, 1)}) == 5, n
    for g in (f, b):
        assert g(dtype=3) == 4
        for bad in (dict(rows=-1), dict(H=0), dict(T=-1), dict(k=0), dict(T=1 << 25, k=4), dict(H=1 << 31),
                    dict(T=1 << 20, H=1 << 20), dict(rows=1 << 31)):
            assert g(**bad) == 2, (g, bad)
    assert f(T=0, y=NULL, out=NULL) == 0 and b(T=0, rows=0, y=NULL, d=NULL) == 0


def test_logprobs_refusals(L, p):
    inf, nan = float("inf"), float("nan")

    def f(x=p, dtype=0, ld=100, T=2, V=100, t=p, temp=1.0, n=2, lp=p, H=p, st=p, tl=p, ti=p, ws=NULL, nws=0):
        return L.mxfp8_token_logprobs(x, dtype, ld, T, V, t, temp, n, lp, H, st, tl, ti, ws, nws, NULL)

    def b(x=p, dtype=0, ld=100, T=2, V=100, t=p, st=p, H=p, g=p, h=p, temp=1.0, dx=p, ldo=100):
        return L.mxfp8_token_logprobs_backward(x, dtype, ld, T, V, t, st, H, g, h, temp, dx, ldo, NULL)
    for n in ("x", "t", "lp", "H", "st", "tl", "ti"):
        assert f(**{n: NULL}) == 1 and f(**{n: _off(p, 1)}) == 5, n
    for n in ("x", "t", "st", "H", "dx"):
        assert b(**{n: NULL}) == 1 and b(**{n: _off(p, 1)}) == 5, n
    assert b(g=NULL, h=NULL) == 1 and b(g=_off(p, 2)) == 5 and b(h=_off(p, 2)) == 5
    assert f(ws=_off(p, 8), nws=64) == 5 and f(t=_off(p, 4)) == 5
    for g in (f, b):
        assert g(dtype=2) == 4
        for bad in (dict(T=-1), dict(V=0), dict(ld=99), dict(temp=0.0), dict(temp=-1.0), dict(temp=inf), dict(temp=nan),
                    dict(V=1 << 31, ld=1 << 31), dict(T=1 << 24)):
            assert g(**bad) == 2, (g, bad)
    assert f(n=-1) == 2 and f(n=65) == 2 and f(V=1, ld=1, n=2) == 2
    assert b(ldo=99) == 2 and b(ld=104) == 2                            # in place, but other strides
    assert f(T=0, x=NULL) == 0 and b(T=0, x=NULL) == 0


def test_python_checks():
    x, ids, w = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for call in (lambda: m.route(x, 2), lambda: m.route_backward(x, ids, w), lambda: m.route_tables(ids, 8),
                 lambda: m.moe_combine(x, ids, w), lambda: m.moe_combine_backward(x, x, ids, w, ids),
                 lambda: m.token_logprobs(x, torch.zeros(4, dtype=torch.int64)),
                 lambda: m.token_logprobs_backward(x, torch.zeros(4, dtype=torch.int64), w, None, None)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(TypeError):
        m.route(x.half(), 2)
    with pytest.raises(TypeError):
        m.token_logprobs([1.0], None)
