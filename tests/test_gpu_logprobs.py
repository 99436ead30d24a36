"""Token log-probabilities, entropy, top alternatives and their gradient
against fp64."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
INF = float("inf")


def _inputs(T, V, dtype, seed, scale=2.0, masked=True):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn((T, V), generator=g, device="cuda") * scale
    x[torch.arange(T), torch.randint(0, V, (T,), generator=g, device="cuda")] += 9.0
    if masked and V > 20:
        x[:, V - V // 10:] = -INF
    t = torch.randint(0, max(1, V - V // 10), (T,), generator=g, device="cuda")
    t[::5] = -100
    return x.to(dtype), t


def _exact(x, t, temp):
    z = x.double() / temp
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    s = e.sum(1, keepdim=True)
    L = torch.log(s)
    logp = z - m - L
    p = e / s
    plogp = torch.where(p > 0, p * logp, torch.zeros_like(p))
    lp = torch.where(t >= 0, logp.gather(1, t.clamp_min(0).unsqueeze(1)).squeeze(1), torch.zeros_like(t, dtype=torch.float64))
    far = torch.where(p > 0, p * (z - m).abs(), torch.zeros_like(p)).sum(1)         # mean distance from the maximum
    return z, m.squeeze(1), L.squeeze(1), logp, p, lp, -plogp.sum(1), far


def _adds(V):
    # a thread adds at most V / 256 terms one after the other, then lanes, waves and slices join
    return V / 256 + 6 + 4 + 64


def _check(mx, x, t, temp=1.0, n=0):
    r = mx.token_logprobs(x, t, temperature=temp, top_n=n)
    z, m, L, logp, p, lp, H, far = _exact(x, t, temp)
    V = x.shape[1]
    # sum: its additions, and per term the rounded distance, the rounded factor and the product (3 half steps of the
    # distance) and 2^x
    sum_tol = U * (_adds(V) + 4 + 4 * far)
    assert bool(((r.stats[:, 0].double() - m).abs() <= U * m.abs()).all())
    assert bool(((r.stats[:, 1].double() - L).abs() <= sum_tol + 2 * U * L.abs()).all()), (r.stats[:, 1] - L).abs().max()
    zt = torch.where(t >= 0, z.gather(1, t.clamp_min(0).unsqueeze(1)).squeeze(1), torch.zeros_like(m))
    lp_tol = sum_tol + U * (zt.abs() + 2 * m.abs() + 4 * L.abs() + 2 * lp.abs())
    assert bool(((r.logprobs.double() - lp).abs() <= lp_tol).all())
    assert bool((r.logprobs[t < 0] == 0).all())
    ent_tol = sum_tol * (1 + 2 * far) + U * (2 * L.abs() + (_adds(V) + 8) * far)
    assert bool(((r.entropy.double() - H).abs() <= ent_tol).all()), ((r.entropy - H).abs() / ent_tol).max()
    if n:
        order = torch.sort(x.double(), dim=1, descending=True, stable=True).indices[:, :n]
        assert r.top_ids.dtype == torch.int64 and torch.equal(r.top_ids, order)
        want = logp.gather(1, order)
        tol = sum_tol.unsqueeze(1) + U * (z.gather(1, order).abs() + 2 * (m + 2 * L).abs().unsqueeze(1) + 2 * want.abs())
        same = want == r.top_logprobs                          # -Inf among them
        assert bool((same | ((r.top_logprobs.double() - want).abs() <= tol)).all())
    else:
        assert r.top_ids is None and r.top_logprobs is None
    return r


CASES = [(1, 1, torch.float32, 1.0, 1), (3, 2, torch.bfloat16, 0.7, 2), (1, 131072, torch.bfloat16, 1.0, 20),
         (2, 100003, torch.float32, 1.3, 64), (5, 1000, torch.bfloat16, 0.7, 5), (37, 4097, torch.float32, 1.0, 1),
         (64, 32000, torch.bfloat16, 1.3, 0), (700, 5001, torch.bfloat16, 1.0, 7), (2100, 1023, torch.float32, 0.7, 3),
         (4, 12289, torch.bfloat16, 1.0, 40), (9, 63, torch.float32, 1.0, 63)]


@pytest.mark.parametrize("T,V,dtype,temp,n", CASES)
def test_logprobs(mx, T, V, dtype, temp, n):
    x, t = _inputs(T, V, dtype, T + V)
    _check(mx, x, t, temp, n)


def test_logprobs_ties(mx):
    # equal logits: the lower column first, whichever wave or slice meets it
    x = torch.zeros((3, 70000), device="cuda", dtype=torch.bfloat16)
    t = torch.tensor([0, 69999, -1], device="cuda")
    r = _check(mx, x, t, n=33)
    assert torch.equal(r.top_ids, torch.arange(33, device="cuda").repeat(3, 1))
    x[1, 5::7] = 1.0
    _check(mx, x, t, n=33)
    _check(mx, torch.randint(0, 3, (300, 9001), device="cuda").bfloat16(), torch.zeros(300, dtype=torch.int64, device="cuda"), n=9)


def test_logprobs_masked_rows(mx):
    low = torch.finfo(torch.float32).min
    for V in (50, 9000):
        x, t = _inputs(6, V, torch.float32, 3, masked=False)
        t = t.clamp_min(0)
        clean = mx.token_logprobs(x, t, top_n=4)
        x[1] = -INF                                            # nothing can occur
        x[2] = -INF
        x[2, V - 1] = 3.0                                      # one certain token, at the end
        t[2] = V - 1
        x[3] = low                                             # the lowest value everywhere: a uniform row
        x[4, 7] = float("nan")
        r = mx.token_logprobs(x, t, top_n=4)
        for i in (0, 5):
            for a, b in ((r.logprobs, clean.logprobs), (r.entropy, clean.entropy), (r.stats, clean.stats),
                         (r.top_ids, clean.top_ids), (r.top_logprobs, clean.top_logprobs)):
                assert torch.equal(a[i], b[i])
        assert r.stats[1, 0] == -INF and torch.isnan(r.stats[1, 1]) and torch.isnan(r.logprobs[1]) and torch.isnan(r.entropy[1])
        assert r.logprobs[2] == 0 and r.entropy[2] == 0 and r.stats[2].tolist() == [3.0, 0.0]
        assert r.top_ids[2].tolist() == [V - 1, 0, 1, 2] and r.top_logprobs[2].tolist() == [0.0, -INF, -INF, -INF]
        assert abs(r.entropy[3].item() - math.log(V)) <= U * (_adds(V) + 8) * math.log(V)
        assert r.top_ids[3].tolist() == [0, 1, 2, 3]
        for a in (r.stats[4], r.logprobs[4:5], r.entropy[4:5], r.top_logprobs[4]):
            assert torch.isnan(a).all()
        assert int(r.top_ids.min()) >= 0 and int(r.top_ids.max()) < V
        d = mx.token_logprobs_backward(x, t, r.stats, r.entropy, torch.ones(6, device="cuda"), torch.ones(6, device="cuda"))
        assert torch.all(d[2] == 0)                            # certain: no gradient
        for i in (0, 3, 5):
            assert torch.isfinite(d[i]).all()


def test_logprobs_sharp_and_flat_rows(mx):
    x = torch.zeros((4, 3001), device="cuda")
    x[0, 17] = 80.0
    x[1, 3000] = 14.0
    x[2] = torch.linspace(-1e4, 1e4, 3001, device="cuda")
    x[3, :] = 1e-3 * torch.arange(3001, device="cuda")
    t = torch.tensor([17, 0, 3000, 1], device="cuda")
    r = _check(mx, x, t, n=3)
    assert r.logprobs[0] == 0


def test_logprobs_targets_out_of_range_strides_and_streams(mx):
    wide, t = _inputs(12, 5003, torch.bfloat16, 8)
    x = wide[:, 1:4000]
    t = t.clamp(-100, 3000)
    t[3], t[4] = 3999, 1 << 40
    r = mx.token_logprobs(x, t, top_n=3)
    assert r.logprobs[3] == 0 and r.logprobs[4] == 0
    flat = mx.token_logprobs(x.contiguous(), t, top_n=3)
    for a, b in ((r.logprobs, flat.logprobs), (r.entropy, flat.entropy), (r.stats, flat.stats), (r.top_ids, flat.top_ids)):
        assert torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o = mx.token_logprobs(x, t, top_n=3)
    s.synchronize()
    assert torch.equal(o.logprobs, r.logprobs) and torch.equal(o.top_logprobs, r.top_logprobs)
    e = mx.token_logprobs(x[:0], t[:0], top_n=3)
    assert e.logprobs.shape == (0,) and e.top_ids.shape == (0, 3)
    assert mx.token_logprobs_backward(x[:0], t[:0], e.stats, e.entropy, e.logprobs).shape == (0, 3999)


# ------------------------------------------------------------------ gradient

@pytest.mark.parametrize("T,V,dtype,temp,which", [
    (1, 1, torch.float32, 1.0, "gh"), (3, 2, torch.bfloat16, 0.7, "gh"), (9, 1001, torch.float32, 1.3, "gh"),
    (5, 32000, torch.bfloat16, 1.0, "gh"), (7, 100003, torch.float32, 0.7, "g"), (6, 8193, torch.bfloat16, 1.3, "h"),
    (300, 515, torch.float32, 1.0, "gh")])
def test_logprobs_backward(mx, T, V, dtype, temp, which):
    x, t = _inputs(T, V, dtype, T * V)
    r = mx.token_logprobs(x, t, temperature=temp)
    gen = torch.Generator("cuda").manual_seed(4)
    g = torch.randn(T, generator=gen, device="cuda") if "g" in which else None
    h = torch.randn(T, generator=gen, device="cuda") if "h" in which else None
    d = mx.token_logprobs_backward(x, t, r.stats, r.entropy, g, h, temperature=temp)
    z, m, L, logp, p, lp, H, far = _exact(x, t, temp)
    gd = (torch.zeros(T, device="cuda") if g is None else g).double()
    gd = torch.where(t >= 0, gd, torch.zeros_like(gd)).unsqueeze(1)
    hd = (torch.zeros(T, device="cuda") if h is None else h).double().unsqueeze(1)
    hot = torch.zeros_like(p)
    hot[torch.arange(T), t.clamp_min(0)] = 1
    flogp = torch.where(p > 0, logp, torch.zeros_like(p))
    want = (gd * (hot - p) - hd * p * (flogp + H.unsqueeze(1))) / temp
    size = (gd.abs() * (hot + p) + hd.abs() * p * (flogp.abs() + H.unsqueeze(1))) / temp
    # p: the stored statistics, the distance and the exponent's product; entropy as stored
    stat = U * (_adds(V) + 8 + 4 * far + m.abs() + 4 * L.abs()).unsqueeze(1)
    rel = stat * (1 + far.unsqueeze(1)) + U * (8 + 2 * torch.where(p > 0, z, torch.zeros_like(p)).abs() + 4 * flogp.abs())
    err = (d.double() - want).abs()
    ent = hd.abs() * p / temp * (stat * (1 + 2 * far.unsqueeze(1)) + U * (_adds(V) + 8) * far.unsqueeze(1))
    assert d.dtype == dtype
    assert bool((err <= rel * size + ent + HALF[dtype] * (want.abs() + rel * size) + 1e-37).all()), (err / (rel * size + 1e-37)).max()
    assert bool((d[:, V - V // 10:] == 0).all()) or V <= 20
    # in place, and into strided rows
    buf = torch.zeros((T, V + 3), dtype=dtype, device="cuda")
    mx.token_logprobs_backward(x, t, r.stats, r.entropy, g, h, temperature=temp, out=buf[:, 1:V + 1])
    assert torch.equal(buf[:, 1:V + 1], d) and torch.all(buf[:, 0] == 0) and torch.all(buf[:, V + 1:] == 0)
    y = x.clone()
    assert mx.token_logprobs_backward(y, t, r.stats, r.entropy, g, h, temperature=temp, out=y) is y
    assert torch.equal(y, d)


def test_logprobs_backward_differences(mx):
    x, t = _inputs(3, 30, torch.float32, 77, masked=False)
    t = t.clamp_min(0)
    g, h = torch.tensor([1.0, -0.5, 0.0], device="cuda"), torch.tensor([0.3, 0.0, -1.0], device="cuda")
    r = mx.token_logprobs(x, t, temperature=0.7)
    d = mx.token_logprobs_backward(x, t, r.stats, r.entropy, g, h, temperature=0.7).double()
    x0, step = x.double(), 1e-5

    def f(v):
        _, _, _, _, _, lp, H, _ = _exact(v, t, 0.7)
        return g.double() * lp + h.double() * H
    for c in range(30):
        a, b = x0.clone(), x0.clone()
        a[:, c] += step
        b[:, c] -= step
        # differences: step^2 / 6 of the third derivative (below 100), 2^-52 * 40 / step of rounding
        torch.testing.assert_close(d[:, c], (f(a) - f(b)) / (2 * step), rtol=0, atol=5e-6)


def test_logprobs_long_offsets(mx):
    # rows beyond 2^31 elements: 40 rows of bf16, 2^26 apart
    T, ld, V = 40, 1 << 26, 2001
    store = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(store, (T, V), (ld, 1))
    src, t = _inputs(T, V, torch.bfloat16, 6)
    x.copy_(src)
    a, b = mx.token_logprobs(x, t, top_n=3), mx.token_logprobs(src, t, top_n=3)
    assert torch.equal(a.logprobs, b.logprobs) and torch.equal(a.top_ids, b.top_ids)
    g = torch.ones(T, device="cuda")
    d = mx.token_logprobs_backward(src, t, b.stats, b.entropy, g, g)
    mx.token_logprobs_backward(x, t, a.stats, a.entropy, g, g, out=x)
    assert torch.equal(x, d)


def test_logprobs_checks(mx):
    x, t = _inputs(4, 64, torch.float32, 1)
    for bad in (lambda: mx.token_logprobs(x, t[:2]), lambda: mx.token_logprobs(x.t(), t), lambda: mx.token_logprobs(x[0], t),
                lambda: mx.token_logprobs_backward(x, t, t, None, None),
                lambda: mx.token_logprobs_backward(x, t, torch.zeros((4, 2), device="cuda"), None, None, torch.zeros(4, device="cuda")),
                lambda: mx.token_logprobs_backward(x, t, torch.zeros((4, 2), device="cuda"), None, torch.zeros(3, device="cuda")),
                lambda: mx.token_logprobs_backward(x, t, torch.zeros((4, 2), device="cuda"), None, torch.zeros(4, device="cuda"), out=x[:2])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: mx.token_logprobs(x, t, top_n=65), lambda: mx.token_logprobs(x, t, temperature=0.0)):
        with pytest.raises(mx.MXFP8Error):
            bad()
    with pytest.raises(TypeError):
        mx.token_logprobs(x, t.int())
