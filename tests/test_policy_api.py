"""The calls of include/mxfp8_policy.h without a GPU: the C entry points refuse
bad arguments on the host before any device work, and the Python calls' own
checks."""
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
    from mxfp8_block_scaled_05_amd._policy import policy_lib
    return policy_lib()


class Space:
    """Addresses in host memory, never read: buffers 2^20 bytes apart."""

    def __init__(self):
        self.store = ctypes.create_string_buffer(40 << 20)
        self.base = (ctypes.addressof(self.store) + 63) & ~63

    def __getitem__(self, slot):
        return ctypes.c_void_p(self.base + (slot << 20))


@pytest.fixture(scope="module")
def space():
    return Space()


def off(p, n):
    return ctypes.c_void_p(p.value + n)


def test_library_exports_every_declared_symbol(L):
    src = open(os.path.join(ROOT, "include", "mxfp8_policy.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(mxfp8_[a-z_0-9]+)\s*\(", src)))
    assert len(names) == 8
    for n in names:
        assert hasattr(L, n), n


def _swiglu(L, s, gu=0, ld=128, T=4, I=64, h=1, hq=NULL, hs=NULL, layout=0, q=4, sc=5):
    pick = lambda v: s[v] if isinstance(v, int) else v
    return L.mxfp8_swiglu(pick(gu), ld, T, I, pick(h), pick(hq), pick(hs), layout, pick(q), pick(sc), NULL)


def test_swiglu_refusals(L, space):
    r = lambda **a: _swiglu(L, space, **a)
    fine = r()
    assert fine not in (0, 1, 2, 3, 4, 5, 8)
    assert r(h=NULL, hq=2, hs=3) == fine and r(h=NULL, hq=2, hs=3, layout=1) == fine and r(q=NULL, sc=NULL) == fine
    assert r(T=0) == 0 and r(T=0, gu=NULL) == 0
    for a in (dict(gu=NULL), dict(h=NULL), dict(h=NULL, hq=2), dict(h=NULL, hs=2), dict(hq=2), dict(hs=3), dict(q=NULL), dict(sc=NULL)):
        assert r(**a) == 1, a
    for a in (dict(T=-1), dict(I=0), dict(I=48), dict(I=16), dict(ld=127), dict(ld=120), dict(ld=132), dict(T=1 << 31),
              dict(T=1 << 30, I=32), dict(I=1 << 30, ld=1 << 31, T=1), dict(T=1 << 20, ld=1 << 41)):
        assert r(**a) == 2, a
    assert r(T=1 << 20, I=1 << 14, ld=1 << 15, layout=1, h=NULL, hq=2, hs=3, q=NULL, sc=NULL) not in (0, 1, 3, 4, 5)
    assert r(layout=2) == 4 and r(layout=-1) == 4
    for name in ("gu", "h", "q", "sc"):
        assert r(**{name: off(space[{"gu": 0, "h": 1, "q": 4, "sc": 5}[name]], 8)}) == 5, name
    assert r(h=NULL, hq=off(space[2], 4), hs=3) == 5 and r(h=NULL, hq=2, hs=off(space[3], 1)) == 5


def test_swiglu_overlap(L, space):
    r = lambda **a: _swiglu(L, space, **a)
    fine = r()
    at = lambda slot, n: off(space[slot], n)
    # gu: 4 rows of 256 bytes; h 512; saved 512 + 16
    assert r(h=0) == 8 and r(h=at(0, 1008)) == 8 and r(h=at(0, 1024)) == fine and r(h=at(0, -512)) == fine
    assert r(q=0) == 8 and r(sc=at(0, 1008)) == 8 and r(sc=at(0, 1024)) == fine
    assert r(h=4) == 8 and r(sc=at(4, 496)) == 8 and r(sc=at(4, 512)) == fine and r(h=5) == 8
    assert r(h=NULL, hq=2, hs=2) == 8 and r(h=NULL, hq=2, hs=at(2, 256)) == fine
    assert r(h=NULL, hq=2, hs=at(2, 256), layout=1) == 8            # packed: whole panels of 256 rows
    # between strided rows
    assert r(ld=256, h=at(0, 256), T=1) == fine and r(ld=256, sc=at(0, 256)) == fine and r(ld=256, sc=at(0, 248)) == 5


def _swiglu_back(L, s, d=0, ld=64, T=4, I=64, q=1, sc=2, dg=3, h=4):
    pick = lambda v: s[v] if isinstance(v, int) else v
    return L.mxfp8_swiglu_backward(pick(d), ld, T, I, pick(q), pick(sc), pick(dg), pick(h), NULL)


def test_swiglu_backward_refusals(L, space):
    r = lambda **a: _swiglu_back(L, space, **a)
    fine = r()
    assert fine not in (0, 1, 2, 3, 4, 5, 8)
    assert r(h=NULL) == fine and r(h=0) == fine and r(T=0, d=NULL) == 0
    for a in (dict(d=NULL), dict(q=NULL), dict(sc=NULL), dict(dg=NULL)):
        assert r(**a) == 1, a
    for a in (dict(T=-1), dict(I=0), dict(I=40), dict(ld=56), dict(ld=68), dict(h=0, ld=72)):
        assert r(**a) == 2, a
    for i, name in enumerate(("d", "q", "sc", "dg", "h")):
        assert r(**{name: off(space[i], 8)}) == 5, name
    assert r(dg=0) == 8 and r(dg=1) == 8 and r(dg=off(space[2], -16)) == 8 and r(h=3) == 8 and r(h=off(space[0], 16)) == 8
    assert r(h=1) == 8


def test_swiglu_python_checks():
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    for bad, error in ((x, ValueError), (x.float(), (TypeError, ValueError)), ("x", TypeError)):
        with pytest.raises(error):
            m.swiglu(bad)
    with pytest.raises(ValueError):
        m.swiglu_backward(x, x, x)


# ------------------------------------------------------------------ adapters

def _lora(L, s, y=0, ydt=1, ldy=64, x=1, ldx=96, T=4, a=2, b=3, sc=4, E=2, r=8, K=96, N=64, off_=5, tok=6, rows=64, hid=7, ws=8,
          bytes_=None):
    pick = lambda v: s[v] if isinstance(v, int) else v
    need = L.mxfp8_lora_add_workspace_bytes(rows, E, r, K, N)
    return L.mxfp8_lora_add(pick(y), ydt, ldy, pick(x), ldx, T, pick(a), pick(b), pick(sc), E, r, K, N, pick(off_), pick(tok), rows,
                            pick(hid), pick(ws), need if bytes_ is None else bytes_, NULL)


BAD_SIZES = (dict(rows=33), dict(rows=-32), dict(E=0), dict(E=1025), dict(r=0), dict(r=4), dict(r=12), dict(r=136), dict(K=0), dict(K=100),
             dict(N=0), dict(N=60), dict(K=1 << 31), dict(rows=1 << 31), dict(rows=1 << 29, N=1 << 20))


def test_lora_add_refusals(L, space):
    r = lambda **a: _lora(L, space, **a)
    fine = r()
    assert fine not in (0, 1, 2, 3, 4, 5, 8)
    assert r(sc=NULL) == fine and r(hid=NULL) == fine and r(ydt=0) == fine and r(T=0, x=NULL, y=NULL) == fine
    assert r(rows=0, bytes_=0) == 0
    for a in (dict(y=NULL), dict(x=NULL), dict(a=NULL), dict(b=NULL), dict(off_=NULL), dict(tok=NULL), dict(ws=NULL)):
        assert r(**a) == 1, a
    for a in BAD_SIZES + (dict(T=-1), dict(T=1 << 31), dict(ldy=56), dict(ldy=68), dict(ldx=88), dict(ldx=100), dict(bytes_=0),
                          dict(T=1 << 20, ldx=1 << 41)):
        assert r(**a) == 2, a
    assert r(ydt=2) == 4 and r(ydt=-1) == 4
    for name, slot in (("y", 0), ("x", 1), ("a", 2), ("b", 3), ("hid", 7), ("ws", 8)):
        assert r(**{name: off(space[slot], 8)}) == 5, name
    assert r(sc=off(space[4], 2)) == 5 and r(off_=off(space[5], 1)) == 5 and r(tok=off(space[6], 4)) == 5


def test_lora_workspaces(L):
    f, g = L.mxfp8_lora_add_workspace_bytes, L.mxfp8_lora_backward_workspace_bytes
    base = dict(rows=64, E=2, r=8, K=96, N=64)
    assert f(*base.values()) >= 64 * 8 * 4 and g(*base.values()) > f(*base.values())
    for a in BAD_SIZES:
        assert f(*dict(base, **a).values()) == 0 and g(*dict(base, **a).values()) == 0, a


def test_lora_add_overlap(L, space):
    r = lambda **a: _lora(L, space, **a)
    fine = r()
    need = L.mxfp8_lora_add_workspace_bytes(64, 2, 8, 96, 64)
    sizes = {"y": 4 * 128, "hid": 64 * 32, "ws": need}
    at = {"y": 0, "x": 1, "a": 2, "b": 3, "sc": 4, "off_": 5, "tok": 6, "hid": 7, "ws": 8}
    length = dict(sizes, x=4 * 192, a=2 * 8 * 96 * 2, b=2 * 64 * 8 * 2, sc=8, off_=12, tok=512)
    for out in ("y", "hid", "ws"):
        for other in at:
            if other == out:
                continue
            assert r(**{out: space[at[other]]}) == 8, (out, other)
            assert r(**{out: off(space[at[other]], -sizes[out] // 16 * 16)}) == fine, (out, other)
            assert r(**{out: off(space[at[other]], (length[other] + 15) // 16 * 16)}) == fine, (out, other)
    # x and y rows in one buffer, side by side and not
    assert r(x=space[0], ldx=160, y=off(space[0], 192), ldy=160) == fine
    assert r(x=space[0], ldx=160, y=off(space[0], 176), ldy=160) == 8


def _back(L, s, dx=0, lddx=96, dy=1, lddy=64, x=2, xs=NULL, form=0, ldx=96, T=4, a=3, b=4, sc=5, E=2, r=8, K=96, N=64, off_=6, tok=7,
          rows=64, hid=8, da=9, db=10, ws=12, bytes_=None):
    pick = lambda v: s[v] if isinstance(v, int) else v
    need = L.mxfp8_lora_backward_workspace_bytes(rows, E, r, K, N)
    return L.mxfp8_lora_backward(pick(dx), lddx, pick(dy), lddy, pick(x), pick(xs), form, ldx, T, pick(a), pick(b), pick(sc), E, r, K, N,
                                 pick(off_), pick(tok), rows, pick(hid), pick(da), pick(db), pick(ws),
                                 need if bytes_ is None else bytes_, NULL)


def test_lora_backward_refusals(L, space):
    r = lambda **a: _back(L, space, **a)
    fine = r()
    assert fine not in (0, 1, 2, 3, 4, 5, 8)
    assert r(dx=NULL) == fine and r(dx=NULL, lddx=0) == fine and r(sc=NULL) == fine
    assert r(form=1, xs=11) == fine and r(form=2, xs=11, ldx=0) == fine
    assert r(T=0, dy=NULL, x=NULL, tok=NULL, hid=NULL) == fine and r(rows=0, dy=NULL, x=NULL, tok=NULL, hid=NULL) == fine
    for a in (dict(dy=NULL), dict(x=NULL), dict(a=NULL), dict(b=NULL), dict(off_=NULL), dict(tok=NULL), dict(hid=NULL), dict(da=NULL),
              dict(db=NULL), dict(ws=NULL), dict(form=1), dict(form=2)):
        assert r(**a) == 1, a
    for a in BAD_SIZES + (dict(T=-1), dict(T=1 << 31), dict(lddx=88), dict(lddx=100), dict(lddy=56), dict(lddy=66), dict(ldx=88), dict(ldx=100),
                          dict(form=1, xs=11, K=104, ldx=104, lddx=104), dict(form=2, xs=11, K=40, lddx=96), dict(bytes_=100)):
        assert r(**a) == 2, a
    assert r(form=3) == 4 and r(form=-1) == 4
    for name, slot in (("dx", 0), ("dy", 1), ("x", 2), ("a", 3), ("b", 4), ("hid", 8), ("da", 9), ("db", 10), ("ws", 12)):
        assert r(**{name: off(space[slot], 8)}) == 5, name
    assert r(form=1, xs=off(space[11], 8)) == 5
    assert r(sc=off(space[5], 1)) == 5 and r(off_=off(space[6], 2)) == 5 and r(tok=off(space[7], 4)) == 5


def test_lora_backward_overlap(L, space):
    r = lambda **a: _back(L, space, **a)
    fine = r()
    at = {"dx": 0, "dy": 1, "x": 2, "a": 3, "b": 4, "sc": 5, "off_": 6, "tok": 7, "hid": 8, "da": 9, "db": 10, "ws": 12}
    for out in ("dx", "da", "db", "ws"):
        for other in at:
            if other != out:
                assert r(**{out: space[at[other]]}) == 8, (out, other)
    assert r(form=1, xs=11, da=off(space[11], -16)) == 8 and r(form=1, xs=11, da=off(space[11], 16)) == fine
    assert r(form=2, xs=11, da=off(space[11], 512)) == 8              # packed: the whole panel's scales
    assert r(form=2, xs=11, db=off(space[2], 1 << 14)) == 8


# ------------------------------------------------------------------ drafts

def _drafts(L, s, x=0, dt=0, ld=100, R=6, V=100, off_=1, B=2, ids=2, u=3, d=4, ldd=100, noise=5, ldn=100, t=1.0, acc=6, tok=7, lp=8, ws=9,
            bytes_=None):
    pick = lambda v: s[v] if isinstance(v, int) else v
    need = L.mxfp8_verify_drafts_workspace_bytes(R, B, V, d is not NULL)
    return L.mxfp8_verify_drafts(pick(x), dt, ld, R, V, pick(off_), B, pick(ids), pick(u), pick(d), ldd, pick(noise), ldn, t, pick(acc),
                                 pick(tok), pick(lp), pick(ws), need if bytes_ is None else bytes_, NULL)


def test_verify_drafts_refusals(L, space):
    r = lambda **a: _drafts(L, space, **a)
    fine = r()
    assert fine not in (0, 1, 2, 3, 4, 5, 8)
    assert r(d=NULL) == fine and r(dt=1) == fine and r(R=2, ids=NULL, u=NULL, d=NULL) == fine and r(d=NULL, ldd=0) == fine
    assert r(B=0, bytes_=0) == 0 and r(t=2.0 ** -60) == fine and r(t=2.0 ** 60) == fine
    for name in ("x", "off_", "ids", "u", "noise", "acc", "tok", "lp", "ws"):
        assert r(**{name: NULL}) == 1, name
    nan = float("nan")
    for a in (dict(R=1), dict(R=-1, B=-1), dict(B=-1), dict(V=0), dict(V=1 << 31, ld=1 << 31), dict(ld=99), dict(ldd=99), dict(ldn=99),
              dict(R=1 << 31), dict(R=1 << 22), dict(t=0.0), dict(t=-1.0), dict(t=nan), dict(t=2.0 ** 61), dict(bytes_=1),
              dict(ld=1 << 60)):
        assert r(**a) == 2, a
    need = L.mxfp8_verify_drafts_workspace_bytes(6, 2, 100, 1)
    assert need > L.mxfp8_verify_drafts_workspace_bytes(6, 2, 100, 0) > 0 and r(bytes_=need - 1) == 2
    assert L.mxfp8_verify_drafts_workspace_bytes(1, 2, 100, 0) == L.mxfp8_verify_drafts_workspace_bytes(0, 0, 100, 0) == 0
    assert r(dt=2) == 4 and r(dt=-1) == 4
    for name, slot, n in (("x", 0, 2), ("off_", 1, 2), ("ids", 2, 4), ("u", 3, 2), ("d", 4, 2), ("noise", 5, 2), ("acc", 6, 2), ("tok", 7, 4),
                          ("lp", 8, 2), ("ws", 9, 8)):
        assert r(**{name: off(space[slot], n)}) == 5, name
    assert r(dt=1, x=off(space[0], 2)) == fine and r(dt=1, x=off(space[0], 1)) == 5


def test_verify_drafts_overlap(L, space):
    r = lambda **a: _drafts(L, space, **a)
    fine = r()
    at = {"x": 0, "off_": 1, "ids": 2, "u": 3, "d": 4, "noise": 5, "acc": 6, "tok": 7, "lp": 8, "ws": 9}
    for out in ("acc", "tok", "lp", "ws"):
        for other in at:
            if other != out:
                assert r(**{out: space[at[other]]}) == 8, (out, other)
    assert r(acc=off(space[0], 2392)) == 8 and r(acc=off(space[0], 2400)) == fine
    assert r(ld=200, acc=off(space[0], 400)) == fine and r(ld=200, lp=off(space[0], 384)) == 8


def test_adapter_and_draft_python_checks():
    b16 = lambda *n: torch.zeros(n, dtype=torch.bfloat16)
    with pytest.raises((TypeError, ValueError)):
        m.lora_add_(b16(4, 64), b16(4, 96), b16(2, 8, 96), b16(2, 64, 8), None)
    with pytest.raises((TypeError, ValueError)):
        m.verify_drafts(torch.zeros(4, 9), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.long), torch.zeros(2),
                        torch.zeros(2, 9))
