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
    assert len(names) >= 2
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
