"""The likeliest columns of rows whose order is hard to find: sorted, tied,
masked, with the best of them in one thread's columns, and lists as long as
the row."""
import pytest
import torch

pytestmark = pytest.mark.gpu

INF = float("inf")


def _check(mx, x, n, what):
    """ids: the stable order; log-probabilities against fp64.  They are x - max - log sum: each of the fp32
    statistics is off by a few half steps of itself, the rounding of the result by half a step of its size."""
    print("top", what, tuple(x.shape), x.dtype, n, flush=True)
    T, V = x.shape
    r = mx.token_logprobs(x, torch.zeros(T, dtype=torch.int64, device="cuda"), top_n=n)
    want = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :n]
    assert torch.equal(r.top_ids, want), what
    z = x.double()
    lp = torch.gather(z - torch.logsumexp(z, 1, keepdim=True), 1, want)
    ok = torch.isfinite(lp)
    assert torch.equal(torch.isfinite(r.top_logprobs), ok)
    # the sum: fewer than 2^11 additions a thread and 10 joins, each half a step
    tol = 2.0 ** -24 * (lp.abs() + 32 + 2.0 ** 11 * 2.0 ** -5)
    assert torch.all((r.top_logprobs.double() - lp)[ok].abs() <= tol[ok]), what


@pytest.mark.parametrize("T,V,n", [(1, 131072, 64), (3, 70001, 20), (300, 9001, 5), (300, 40000, 64), (257, 600001, 3),
                                   (5, 1, 1), (9, 20, 20), (400, 64, 64), (2, 2100000, 20), (260, 33000, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_hard_orders(mx, T, V, n, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(V + n)
    x = (torch.randn((T, V), generator=g, device="cuda") * 2).to(dtype)
    _check(mx, x, n, "random")
    up = torch.linspace(-3, 3, V, device="cuda").to(dtype).expand(T, V).contiguous()
    _check(mx, up, n, "rising")
    _check(mx, up.flip(1).contiguous(), n, "falling")
    _check(mx, torch.full((T, V), 0.25, dtype=dtype, device="cuda"), n, "equal")
    few = torch.randint(-2, 2, (T, V), generator=g, device="cuda").to(dtype)
    _check(mx, few, n, "four values")
    y = x.clone()
    y[:, V // 3:] = -INF
    _check(mx, y, n, "masked from a third on")
    y = torch.full_like(x, -INF)
    y[:, V - 1] = 1.0
    _check(mx, y, n, "one column left")
    y = torch.full_like(x, torch.finfo(dtype).min)
    y[:, ::max(1, V // 3)] = x[:, ::max(1, V // 3)]
    _check(mx, y, n, "the type's lowest value")
    y = x.clone()
    y[:, V // 2:V // 2 + 100] += 50                         # the best lie next to each other
    _check(mx, y, n, "neighbours")


def test_nan_rows_give_columns(mx):
    x = torch.randn((4, 5000), device="cuda")
    x[1] = float("nan")
    x[2, 77] = float("nan")
    x[3] = -float("nan")
    r = mx.token_logprobs(x, torch.zeros(4, dtype=torch.int64, device="cuda"), top_n=20)
    for row in r.top_ids.tolist():
        assert len(set(row)) == 20 and min(row) >= 0 and max(row) < 5000
    assert torch.isnan(r.top_logprobs[1:]).all() and torch.isfinite(r.top_logprobs[0]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V", [(2, 9000), (300, 20000), (1100, 700)])
def test_zeros_of_both_signs_are_equal(mx, T, V, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    x = torch.where(torch.rand((T, V), generator=g, device="cuda") < 0.5, -0.0, 0.0).to(dtype)
    x[: T // 2, ::3] = -2.0
    _check(mx, x, 9, "zeros")
