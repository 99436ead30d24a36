"""Renormalized router weights, and their gradient, where the chosen scores are
too small for fp32: their quotients are not."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

HALF32 = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
# an exponential 4 half steps, 1 + e, a quotient; the sum of up to 32 of them 6 additions; the quotient, the scale
TOL = 48 * HALF32


def _weights(z, i, score):
    """fp64 weights over their sum, from the chosen logits alone, and 1 - s of them."""
    a = np.take_along_axis(z, i, 1)
    top = a.max(1, keepdims=True)
    e = np.exp(a - top)
    if score == "sigmoid":
        e = e / (1 + np.exp(a))
        return e / e.sum(1, keepdims=True), 1 / (1 + np.exp(a))
    return e / e.sum(1, keepdims=True), np.ones_like(e)


def _check(mx, x, k, score, bias=None, scale=2.5):
    T = x.shape[0]
    ids, w = mx.route(x, k, score=score, bias=bias, scale=scale)
    z, i = x.double().cpu().numpy(), ids.long().cpu().numpy()
    assert all(len(set(r)) == k for r in i.tolist()) and i.min() >= 0 and i.max() < x.shape[1]
    want, rest = _weights(z, i, score)
    # 2^-126: what fp32 has no normal number for may be 0
    assert np.all(np.abs(w.double().cpu().numpy() - want * scale) <= TOL * want * scale + scale * 2.0 ** -126)
    dw = torch.randn((T, k), device="cuda", generator=torch.Generator("cuda").manual_seed(k))
    d = mx.route_backward(x, ids, dw, score=score, scale=scale).double().cpu().numpy()
    g = dw.double().cpu().numpy() * scale
    full, bound = np.zeros_like(z), np.zeros_like(z)
    mean, size = (g * want).sum(1, keepdims=True), (np.abs(g) * want).sum(1, keepdims=True)
    np.put_along_axis(full, i, (g - mean) * want * rest, 1)
    np.put_along_axis(bound, i, (np.abs(g) + size) * want * rest, 1)
    if score == "softmax":
        # experts that were not chosen: their score times a sum of k terms that cancel
        s = np.exp(z - z.max(1, keepdims=True))
        bound += s / s.sum(1, keepdims=True) * size
    err = np.abs(d - full)
    assert np.all(err <= 2 * TOL * bound + HALF[x.dtype] * np.abs(full) + 1e-37), (err / (2 * TOL * bound + 1e-37)).max()
    return ids, w, d


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(16, 2), (64, 8), (256, 8), (512, 32)])
def test_sigmoid_weights_of_low_logits(mx, E, k, dtype):
    g = torch.Generator("cuda").manual_seed(E)
    noise = torch.randn((12, E), generator=g, device="cuda")
    level = torch.tensor([0, -40, -60, -69, -70, -75, -86, -88, -90, -104, -200, -600], device="cuda").float()
    print("low", E, k, dtype, flush=True)
    ids, w, d = _check(mx, (noise + level.unsqueeze(1)).to(dtype), k, "sigmoid")
    # rows beside them are untouched
    x = (noise + level.unsqueeze(1)).to(dtype)[:5].contiguous()
    ids5, w5 = mx.route(x, k, score="sigmoid", scale=2.5)
    assert torch.equal(ids[:5], ids5) and torch.equal(w[:5], w5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(16, 2), (64, 8), (256, 8), (512, 31)])
def test_softmax_weights_of_experts_far_below_the_largest(mx, E, k, dtype):
    print("far", E, k, dtype, flush=True)
    g = torch.Generator("cuda").manual_seed(E)
    x = torch.randn((10, E), generator=g, device="cuda")
    gap = torch.tensor([0, 40, 60, 69, 75, 87, 90, 104, 150, 600], device="cuda").float()
    x[:, 0] = gap                                                       # an expert that the bias shuts out
    bias = torch.zeros(E, device="cuda")
    bias[0] = -10.0
    ids, _, _ = _check(mx, x.to(dtype), k, "softmax", bias)
    assert not bool((ids == 0).any())


def test_nothing_chosen_has_a_score(mx):
    inf = float("inf")
    x = torch.full((4, 32), -inf, device="cuda")
    x[1, 0] = 1.0                                                       # shut out by the bias
    x[2, 3] = -300.0                                                    # one score, too small for fp32
    x[3] = torch.linspace(-1, 1, 32, device="cuda")
    bias = torch.zeros(32, device="cuda")
    bias[0] = -inf
    for score in ("sigmoid", "softmax"):
        ids, w = mx.route(x, 4, score=score, bias=bias)
        assert torch.isnan(w[0]).all() and torch.isnan(w[1]).all() and torch.isfinite(w[3]).all()
        assert ids[2].tolist() == [3, 1, 2, 4] and w[2].tolist() == [1, 0, 0, 0]
        d = mx.route_backward(x, ids, torch.ones_like(w), score=score)
        assert torch.isnan(d[0].gather(0, ids[0].long())).all() and torch.isnan(d[1].gather(0, ids[1].long())).all()
        assert torch.isfinite(d[2:]).all()
