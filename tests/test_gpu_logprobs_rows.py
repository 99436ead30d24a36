"""The gradient of log-probability and entropy on rows without statistics: a NaN
or +Inf among the logits, or nothing above -Inf."""
import pytest
import torch

pytestmark = pytest.mark.gpu

INF = float("inf")


def _rows(V, dtype):
    """(logits, targets, rows without statistics): the others are ordinary ones."""
    g = torch.Generator("cuda").manual_seed(V)
    x = (torch.randn((9, V), generator=g, device="cuda") * 2).to(dtype)
    t = torch.randint(0, V, (9,), generator=g, device="cuda")
    clean = x.clone()
    x[1] = -INF
    x[2, V // 2] = float("nan")
    x[3, V - 1] = INF
    x[4, 0] = float("nan")
    t[4] = -100
    x[6] = float("nan")
    x[7] = -INF
    t[7] = -100
    x[8, : V // 2] = -INF
    clean[8] = x[8]
    t[8] = V - 1
    return x, clean, t, [1, 2, 3, 4, 6, 7]


@pytest.mark.parametrize("V", [3, 50, 1001, 9000, 20000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("temp", [1.0, 0.7, 1.3])
def test_rows_without_statistics(mx, V, dtype, temp):
    print("rows", V, dtype, temp, flush=True)
    x, clean, t, broken = _rows(V, dtype)
    fine = [i for i in range(9) if i not in broken]
    r = mx.token_logprobs(x, t, temperature=temp)
    rc = mx.token_logprobs(clean, t, temperature=temp)
    assert torch.isnan(r.stats[broken, 1]).all() and torch.isfinite(r.stats[fine]).all()
    one, zero = torch.ones(9, device="cuda"), torch.zeros(9, device="cuda")
    for g, h in ((one, None), (one, zero), (None, one), (None, zero), (one, one), (zero, None), (zero, zero)):
        kw = dict(temperature=temp)
        d = mx.token_logprobs_backward(x, t, r.stats, r.entropy, g, h, **kw)
        assert torch.isnan(d[broken]).all(), (g, h)
        want = mx.token_logprobs_backward(clean, t, rc.stats, rc.entropy, g, h, **kw)
        assert torch.isfinite(want).all() and torch.equal(d[fine], want[fine])
        assert torch.all(d[8, : V // 2] == 0)                           # tokens that cannot occur
        y = x.clone()
        mx.token_logprobs_backward(y, t, r.stats, r.entropy, g, h, out=y, **kw)
        assert torch.equal(y[fine], want[fine]) and torch.isnan(y[broken]).all()
