"""The gated activation with its 8-bit checkpoint on the GPU: the product and its
gradient against fp64, the checkpoint and the product's grids against the
quantizers byte for byte.

Tolerances.  fp32 steps: e^-|g| carries |g| 2^-24 of its value (the rounded
product with log2 e; |g| <= 88 wherever it is not 0, so 2^-17.5), the rest is at
most eight roundings or one-step hardware functions (2^-23 each): 2^-16 of each
term covers both, and a term below 2^-118 of its other factors may be 0.  Then
one rounding to bf16: half a step, 2^-8 of the value (2^-134 among subnormals).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

STEP, FP32 = 2.0 ** -8, 2.0 ** -16
TINY = 2.0 ** -134


def _gu(T, inner, seed=0, spread=3.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((T, 2 * inner), generator=g, device="cuda") * spread
    return torch.where(torch.rand(x.shape, generator=g, device="cuda") < 0.02, x * 10, x).to(torch.bfloat16)


def _near(got, want, terms):
    """got bf16 against want fp64 of terms whose sizes add up to `terms`."""
    off = (got.double() - want).abs()
    ok = off <= STEP * want.abs() + FP32 * terms + TINY
    assert bool(ok.all()), (off - STEP * want.abs() - FP32 * terms).max().item()


def _check_forward(mx, gu, layout="bf16"):
    T, inner = gu.shape[0], gu.shape[1] // 2
    r = mx.swiglu(gu, layout=layout)
    whole = gu.contiguous()
    h = mx.swiglu(gu).h
    g, u = whole.double().chunk(2, 1)
    want = g * torch.sigmoid(g) * u
    _near(h, want, want.abs() + u.abs() * 2.0 ** -102)
    q, s = mx.quantize(whole, 1)
    assert torch.equal(r.saved_q, q) and torch.equal(r.saved_s, s)
    hq, hs = mx.quantize(h, 1)
    if layout == "bf16":
        assert torch.equal(r.h, h)
    elif layout == "canonical":
        assert torch.equal(r.h[0], hq) and torch.equal(r.h[1], hs)
    else:
        w = mx.repack(hq.view(1, T, inner), hs.view(1, T, inner // 32))
        assert torch.equal(r.h.q, w.q) and torch.equal(r.h.s, w.s)


SHAPES = [(1, 32), (1, 768), (3, 96), (33, 768), (255, 160), (257, 128), (64, 4096), (300, 2080), (1000, 416), (16, 12288)]


@pytest.mark.parametrize("layout", ["bf16", "canonical", "packed"])
@pytest.mark.parametrize("T,inner", SHAPES)
def test_forward(mx, T, inner, layout):
    _check_forward(mx, _gu(T, inner, seed=T), layout)


@pytest.mark.parametrize("T,inner", SHAPES)
def test_backward(mx, T, inner):
    gu = _gu(T, inner, seed=T + 1)
    r = mx.swiglu(gu)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    d_h = (torch.randn((T, inner), generator=gen, device="cuda") * 2.0 ** -6).to(torch.bfloat16)
    _check_backward(mx, d_h, r.saved_q, r.saved_s)


def _check_backward(mx, d_h, q, s):
    T, inner = d_h.shape
    d_gu, h = mx.swiglu_backward(d_h, q, s)
    only, none = mx.swiglu_backward(d_h, q, s, recompute=False)
    assert none is None and torch.equal(only, d_gu)
    # autograd of the formula in fp64, at the checkpoint's values
    v = mx.dequantize(q, s, T, 2 * inner, 1, torch.float32).double().requires_grad_(True)
    g, u = v.chunk(2, 1)
    want = torch.nn.functional.silu(g) * u
    (want * d_h.double()).sum().backward()
    sig = torch.sigmoid(g).detach()
    g, u, d = g.detach(), u.detach(), d_h.double()
    size_g = (d * u).abs() * (sig + g.abs() * sig * (1 - sig) + 2.0 ** -102)
    size_u = d.abs() * ((g * sig).abs() + 2.0 ** -102)
    _near(d_gu[:, :inner], v.grad[:, :inner], size_g)
    _near(d_gu[:, inner:], v.grad[:, inner:], size_u)
    _near(h, want.detach(), want.detach().abs() + u.abs() * 2.0 ** -102)


def test_gradient_against_differences(mx):
    """Central differences of the fp64 product at the checkpoint's values: their own error is the step squared times
    the third derivative (at most 0.6 |u| there) over 6, and fp64's rounding over the step."""
    T, inner, step = 40, 64, 1e-4
    r = mx.swiglu(_gu(T, inner, seed=3, spread=1.0))
    d_h = torch.ones((T, inner), dtype=torch.bfloat16, device="cuda")
    d_gu, _ = mx.swiglu_backward(d_h, r.saved_q, r.saved_s)
    g, u = mx.dequantize(r.saved_q, r.saved_s, T, 2 * inner, 1, torch.float32).double().chunk(2, 1)

    def f(x):
        return x * torch.sigmoid(x) * u
    numeric = (f(g + step) - f(g - step)) / (2 * step)
    bound = STEP * numeric.abs() + FP32 * u.abs() * 2 + 0.6 * u.abs() * step ** 2 / 6 + 1e-10 * (1 + (g * u).abs())
    assert bool(((d_gu[:, :inner].double() - numeric).abs() <= bound).all())


def test_extreme_gates(mx):
    """Gates over bf16's range: saturated on both sides, no overflow, exact zeros kept."""
    values = torch.tensor([0.0, -0.0, 1e-38, -1e-38, 88.0, -88.0, 90.0, -90.0, 126.5, -126.5, 1e4, -1e4, 3e38, -3e38, 1.278, -1.278],
                          device="cuda").to(torch.bfloat16)
    gu = torch.zeros((32, 64), dtype=torch.bfloat16, device="cuda")
    gu[:, :16], gu[:, 16:32] = values, values
    gu[:, 32:] = torch.linspace(-1, 1, 32, device="cuda").to(torch.bfloat16).unsqueeze(1)
    _check_forward(mx, gu)
    r = mx.swiglu(gu)
    assert bool(torch.isfinite(r.h).all())
    # one magnitude a block, so the checkpoint keeps each gate
    for v in values.tolist():
        gu[:, :32] = v
        r = mx.swiglu(gu)
        d_h = torch.full((32, 32), 0.5, dtype=torch.bfloat16, device="cuda")
        _check_backward(mx, d_h, r.saved_q, r.saved_s)


def test_nan_and_inf_stay_in_their_blocks(mx):
    gu = _gu(8, 128, seed=9)
    clean = mx.swiglu(gu)
    bad = gu.clone()
    bad[1, 5], bad[2, 128 + 40], bad[3, 70] = float("nan"), float("inf"), float("-inf")
    r = mx.swiglu(bad)
    touched = torch.zeros((8, 128), dtype=torch.bool, device="cuda")
    touched[1, 5] = touched[2, 40] = touched[3, 70] = True
    assert torch.equal(r.h[~touched], clean.h[~touched])
    assert bool(r.h[1, 5].isnan()) and bool(r.h[2, 40].isinf()) and bool(r.h[3, 70].isnan())
    q, s = mx.quantize(bad, 1)
    assert torch.equal(r.saved_q, q) and torch.equal(r.saved_s, s)
    d_h = torch.ones((8, 128), dtype=torch.bfloat16, device="cuda")
    d0, h0 = mx.swiglu_backward(d_h, clean.saved_q, clean.saved_s)
    d1, h1 = mx.swiglu_backward(d_h, r.saved_q, r.saved_s)
    block = torch.zeros((8, 128), dtype=torch.bool, device="cuda")
    block[1, :32] = block[2, 32:64] = block[3, 64:96] = True
    assert bool(h1[block].isnan().all()) and torch.equal(h1[~block], h0[~block])
    both = torch.cat((block, block), 1)
    assert torch.equal(d1[~both], d0[~both])


def test_strided_rows_and_in_place(mx):
    wide = _gu(70, 200, seed=4)
    _check_forward(mx, wide[:, 8:8 + 320])                  # rows 400 apart, inner 160
    r = mx.swiglu(wide[:, 8:8 + 320])
    d = _gu(70, 96, seed=6)
    view = d[:, 16:16 + 160]
    got = mx.swiglu_backward(view, r.saved_q, r.saved_s)
    want = mx.swiglu_backward(view.contiguous(), r.saved_q, r.saved_s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_rows(mx):
    gu = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    r = mx.swiglu(gu)
    assert r.h.shape == (0, 64) and r.saved_q.shape == (0, 128) and r.saved_s.shape == (0, 4)
    d_gu, h = mx.swiglu_backward(r.h, r.saved_q, r.saved_s)
    assert d_gu.shape == (0, 128) and h.shape == (0, 64)
    with pytest.raises(mx.MXFP8Error):
        mx.swiglu(gu, layout="packed")


def test_without_a_checkpoint(mx):
    gu = _gu(50, 96)
    r = mx.swiglu(gu, save=False)
    assert r.saved_q is None and r.saved_s is None and torch.equal(r.h, mx.swiglu(gu).h)


def test_another_stream_and_a_graph(mx):
    a, b = _gu(100, 256, seed=1), _gu(100, 256, seed=2)
    want = [mx.swiglu(t, layout="canonical") for t in (a, b)]
    grads = [mx.swiglu_backward(w.h[0].view(torch.uint8).to(torch.bfloat16), w.saved_q, w.saved_s) for w in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r = mx.swiglu(a, layout="canonical")
    side.synchronize()
    assert torch.equal(r.h[0], want[0].h[0]) and torch.equal(r.saved_q, want[0].saved_q)
    x = a.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = mx.swiglu(x, layout="canonical")
        d_gu, h = mx.swiglu_backward(r.h[0].to(torch.bfloat16), r.saved_q, r.saved_s)
    for i in (0, 1, 0, 1):
        x.copy_((a, b)[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(r.h[0], want[i].h[0]) and torch.equal(r.saved_s, want[i].saved_s)
        assert torch.equal(d_gu, grads[i][0]) and torch.equal(h, grads[i][1])


def test_more_than_2_31_elements(mx):
    """Rows whose offsets pass 32 bits, first and last against a call of those rows alone."""
    inner = 16384
    T = (1 << 31) // (2 * inner) + 40
    gu = torch.empty((T, 2 * inner), dtype=torch.bfloat16, device="cuda")
    for i in range(0, T, 8192):
        gu[i:i + 8192] = _gu(min(8192, T - i), inner, seed=i)
    r = mx.swiglu(gu, layout="canonical")
    d = gu[:, :inner]
    d_gu, h = mx.swiglu_backward(d, r.saved_q, r.saved_s)
    for rows in (slice(0, 20), slice(T - 60, T)):
        part = mx.swiglu(gu[rows], layout="canonical")
        assert torch.equal(part.h[0], r.h[0][rows]) and torch.equal(part.h[1], r.h[1][rows])
        assert torch.equal(part.saved_q, r.saved_q[rows]) and torch.equal(part.saved_s, r.saved_s[rows])
        want = mx.swiglu_backward(d[rows], part.saved_q, part.saved_s)
        assert torch.equal(want[0], d_gu[rows]) and torch.equal(want[1], h[rows])


@pytest.mark.parametrize("layout", ["bf16", "canonical", "packed"])
def test_passes_larger_than_the_last_level_cache(mx, layout):
    """In every form, with and without a checkpoint, against calls of a few rows (which keep to the caches)"""
    T, inner = 1721, 32 * 1223                           # 67 million elements of h: past 256 MB in every form
    gu = _gu(T, inner, seed=4)
    r, bare = mx.swiglu(gu, layout=layout), mx.swiglu(gu, layout=layout, save=False)
    d_h = gu[:, inner:]
    d_gu, h = mx.swiglu_backward(d_h, r.saved_q, r.saved_s)
    alone, none = mx.swiglu_backward(d_h, r.saved_q, r.saved_s, recompute=False)
    assert none is None and torch.equal(alone, d_gu)
    parts = [slice(i, min(i + 256, T)) for i in range(0, T, 256)]
    small = [mx.swiglu(gu[p], layout="bf16" if layout == "bf16" else "canonical") for p in parts]
    assert torch.equal(r.saved_q, torch.cat([s.saved_q for s in small])) and torch.equal(r.saved_s, torch.cat([s.saved_s for s in small]))
    if layout == "bf16":
        want = torch.cat([s.h for s in small])
        assert torch.equal(r.h, want) and torch.equal(bare.h, want)
    else:
        q, s = (torch.cat([part.h[i] for part in small]) for i in (0, 1))
        if layout == "packed":
            w = mx.repack(q.view(1, T, inner), s.view(1, T, inner // 32))
            q, s = w.q, w.s
        for got in (r.h, bare.h):
            a, b = (got.q, got.s) if layout == "packed" else got
            assert torch.equal(a.view(-1), q.view(-1)) and torch.equal(b.view(-1), s.view(-1))
    for p, part in zip(parts, small):
        want = mx.swiglu_backward(d_h[p], part.saved_q, part.saved_s)
        assert torch.equal(d_gu[p], want[0]) and torch.equal(h[p], want[1])
