"""Rows far from 0: of the type's lowest or largest value, also at temperatures
that take them past fp32's range (the distribution is that over the equal
largest logits), and of logits around a common level."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

INF = float("inf")
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.mark.parametrize("V", [7, 1001, 9000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("temp", [1.0, 0.7, 0.5, 1.3, 2.0 ** -20])
def test_rows_of_the_lowest_value(mx, V, dtype, temp):
    print("lowest", V, dtype, temp, flush=True)
    low = torch.finfo(dtype).min
    x = torch.full((6, V), low, dtype=dtype, device="cuda")             # row 0: nothing but the lowest value
    x[1, V // 2:] = -INF                                                # some that cannot occur
    x[2, 3] = 2.0                                                       # one ordinary logit
    x[3, ::2] = -low                                                    # the largest value in every second column
    x[4, 5] = -low
    x[5] = torch.linspace(-3, 3, V, device="cuda").to(dtype)            # an ordinary row beside them
    x[5, 0] = low
    t = torch.tensor([0, 1, 3, 2, -100, 1], device="cuda")
    count = [V, V // 2, 1, (V + 1) // 2, 1]
    r = mx.token_logprobs(x, t, temperature=temp)
    assert torch.isfinite(r.stats).all()
    g = torch.tensor([1.0, -2.0, 0.5, 1.0, 3.0, 1.0], device="cuda")
    h = torch.tensor([0.25, 1.0, -1.0, 0.0, 1.0, 0.5], device="cuda")
    d = mx.token_logprobs_backward(x, t, r.stats, r.entropy, g, h, temperature=temp).double().cpu()
    for i, n in enumerate(count):
        L = math.log(n)
        # log n: the sum of ones is exact, the logarithm off by at most 2 half steps; in stats against the rounded m
        m, z = r.stats[i, 0].item(), x[i].max().item() / temp
        lost = z - m if abs(m) < 2.0 ** 31 else 0.0
        assert abs(r.stats[i, 1].item() - (L + lost)) <= 2 * U * L + 2 * U * abs(lost)
        assert abs(r.entropy[i].item() - L) <= 4 * U * L
        lp = 0.0 if i == 4 else -L
        assert abs(r.logprobs[i].item() - lp) <= 4 * U * L
        p = (x[i] == x[i].max()).double().cpu() / n
        hot = torch.zeros(V, dtype=torch.float64)
        gi, hi = g[i].item(), h[i].item()
        if i == 4:
            gi = 0.0
        else:
            hot[t[i].item()] = 1
        want = gi * (hot - p) / temp                                    # log p + entropy is 0
        # p: half steps of log n (four of its size) and of the exponential's argument and result; the entropy term
        # adds up log p and the entropy, each off by 4 half steps of log n, and the factors' own few
        size = (abs(gi) * (hot + p) + abs(hi) * p * (1 + 2 * L)) / temp
        tol = U * (8 + 8 * L) * size + HALF[dtype] * want.abs() + 1e-37
        assert bool(((d[i] - want).abs() <= tol).all()), (i, (d[i] - want).abs().max())
    assert torch.isfinite(d).all() and d[5, 0] == 0


@pytest.mark.parametrize("temp", [1.0, 0.7, 0.9, 1.3])
@pytest.mark.parametrize("level", [0.0, 300.0, -1e4, 1e6, -1e9, 1e9, -3e9, -1e20, 1e30])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_around_a_level(mx, level, temp, dtype):
    """The gradient's error goes by the distances from the largest logit, not by the logits' own size."""
    print("level", level, temp, dtype, flush=True)
    T, V = 5, 2003
    g = torch.Generator("cuda").manual_seed(9)
    x = (torch.randn((T, V), generator=g, device="cuda", dtype=torch.float64) * 2 + level).to(dtype)
    x[:, -100:] = -INF
    x[1] = level                                                        # equal logits
    t = torch.tensor([0, 1, -100, 700, 1900], device="cuda")
    r = mx.token_logprobs(x, t, temperature=temp)
    gr = torch.tensor([1.0, -2.0, 3.0, 0.5, 1.0], device="cuda")
    h = torch.tensor([0.5, 1.0, -1.0, 0.0, 2.0], device="cuda")
    d = mx.token_logprobs_backward(x, t, r.stats, r.entropy, gr, h, temperature=temp).double()
    xd = x.double()
    top = xd.amax(1, keepdim=True)
    dist = (xd - top) / temp                                            # exact differences, one rounding in fp64
    e = torch.exp(dist)
    L = torch.log(e.sum(1, keepdim=True))
    p, logp = torch.exp(dist - L), torch.where(e > 0, dist - L, torch.zeros_like(e))
    H = -(p * logp).sum(1, keepdim=True)
    gd = torch.where(t >= 0, gr.double(), torch.zeros_like(gr.double())).unsqueeze(1)
    hot = torch.zeros_like(p)
    hot[torch.arange(T), t.clamp_min(0)] = 1
    want = (gd * (hot - p) - h.double().unsqueeze(1) * p * (logp + H)) / temp
    size = (gd.abs() * (hot + p) + h.double().abs().unsqueeze(1) * p * (logp.abs() + H)) / temp
    # what the largest z loses by its rounding: at most half a step, in L's size while |m| < 2^31
    m = (top / temp).abs()
    lost = torch.where(m < 2.0 ** 31, U * m, torch.zeros_like(m))
    far = torch.where(p > 0, p * dist.abs(), torch.zeros_like(p)).sum(1, keepdim=True)
    # half steps: the sum's additions (V / 64 a thread at most, 6 lanes and 4 waves) and its terms' (4 and 4 of the
    # mean distance), L's own four, twice what m lost, the distance's four, the exponential's and the products' 12
    rel = U * (V / 64 + 10 + 4 + 4 * far + 4 * (L + lost) + 2 * lost + 4 * torch.where(p > 0, dist.abs(), torch.zeros_like(p)) + 12)
    rel = rel + 2.0 ** -44 * m * (m < 2.0 ** 31)                        # 1 / temperature in two fp32 parts
    ent = h.double().abs().unsqueeze(1) * p / temp * rel * (1 + 2 * (far + L) + logp.abs())
    tol = rel * size + ent + HALF[dtype] * (want.abs() + rel * size) + 1e-37
    err = (d - want).abs()
    assert bool((err <= tol).all()), (err / tol).max()
    assert bool((d[[0, 2, 3], -100:] == 0).all())
