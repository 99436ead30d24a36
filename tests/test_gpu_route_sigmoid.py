"""The router's sigmoid gradient where the scores are close to 1 or to 0: the
derivative s (1 - s) is held to its own size there."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

HALF32 = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
# a score: the exponential 4 half steps, 1 + e and the quotient; its derivative the same once more; the sum of up to 32
# scores and of their gradients at most 6 additions each, two quotients and a difference, each term twice
TOL = 96 * HALF32


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(16, 1), (64, 8), (300, 31), (512, 32)])
def test_sigmoid_gradient_of_far_logits(mx, E, k, renorm, dtype):
    print("sigmoid", E, k, renorm, dtype, flush=True)
    T = 41
    g = torch.Generator("cuda").manual_seed(E)
    x = ((torch.rand((T, E), generator=g, device="cuda") * 60) - 30).to(dtype)
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).int()
    dw = torch.randn((T, k), generator=g, device="cuda")
    d = mx.route_backward(x, ids, dw, score="sigmoid", renormalize=renorm, scale=2.5).double().cpu().numpy()
    z = x.double().cpu().numpy()
    s, c = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))                    # the score and what it lacks of 1
    rows, i = np.arange(T)[:, None], ids.cpu().numpy()
    a, w = s[rows, i], dw.double().cpu().numpy() * 2.5
    size = np.abs(w)
    if renorm:
        A = a.sum(1, keepdims=True)
        size = size / A + (np.abs(w) * a).sum(1, keepdims=True) / A ** 2
        w = (w - (w * a).sum(1, keepdims=True) / A) / A
    want, bound = np.zeros_like(s), np.zeros_like(s)
    want[rows, i] = w * a * c[rows, i]
    bound[rows, i] = size * a * c[rows, i]
    err = np.abs(d - want)
    assert np.all(err <= TOL * bound + HALF[dtype] * np.abs(want) + 1e-37), (err / (TOL * bound + 1e-37)).max()


def test_sigmoid_gradient_at_the_ends(mx):
    inf = float("inf")
    x = torch.tensor([[inf, -inf, 0.0, 200.0, -200.0, 17.0, -17.0, 1.0]], device="cuda")
    ids = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
    d = mx.route_backward(x, ids, torch.ones((1, 8), device="cuda"), score="sigmoid", renormalize=False)[0].tolist()
    assert d[0] == 0 and d[1] == 0 and abs(d[2] - 0.25) <= 8 * HALF32 and d[3] <= 2e-38 and d[4] <= 2e-38
    want = np.exp(-17.0) / (1 + np.exp(-17.0)) ** 2
    assert abs(d[5] - want) <= TOL * want and abs(d[6] - want) <= TOL * want
