"""The low-rank adapters' fp32 results: A x and S keep all 24 bits in the products
that follow.  Whole numbers, one product for each result, so equality."""
import pytest
import torch

from test_gpu_lora import _by_row, _gen, _ids, _want, _want_grads, _whole

pytestmark = pytest.mark.gpu

# T, E, r, K, N; K and N at most 128, so that sums of 255 * 255 stay below 2^23
WIDE = [(1, 1, 8, 128, 120), (40, 3, 16, 128, 128), (128, 2, 32, 96, 128), (120, 5, 64, 128, 104), (100, 2, 72, 128, 128), (128, 3, 128, 128, 128),
        (9200, 3, 24, 128, 128), (4300, 2, 128, 128, 128)]


def _large(shape, g):
    """Whole numbers of both signs with all of bf16's 8 bits, most of them from 128 on"""
    return torch.randint(100, 256, shape, generator=g, device="cuda")


@pytest.mark.parametrize("T,E,r,K,N", WIDE)
def test_fp32_results_hold_24_bits(mx, T, E, r, K, N):
    """A x and S up to 2^23 and odd: two bf16 numbers would lose their last bits, three hold them all"""
    g = _gen(T + r)
    ids = _ids(T, E, T, none=T > 1)
    tables = mx.route_tables(ids.view(-1, 1), E)
    rank_sign = 1 - 2 * (torch.arange(r, device="cuda") % 2)
    x = _large((T, K), g).to(torch.bfloat16)
    a = (_large((E, r, K), g) * rank_sign.view(1, r, 1)).to(torch.bfloat16)
    # one rank for each column of y
    b = torch.zeros((E, N, r), device="cuda")
    n = torch.arange(N, device="cuda")
    for e in range(E):
        b[e, n, (n * (e + 1) + e) % r] = 1.0 - 2 * (n % 3 == 0)
    b = b.to(torch.bfloat16)
    y = _whole((T, N), g, 1 << 22, torch.float32)
    want, h, _, _ = _want(y, x, a, b, ids, None)
    with_adapter = (ids >= 0).sum().item()
    if with_adapter:
        assert float(h.abs().max()) > 2 ** 19 and float(want.abs().max()) < 2 ** 24 and bool((h % 2 == 1).any())
    hidden = mx.lora_add_(y, x, a, b, tables, keep_hidden=True)
    assert torch.equal(hidden.double(), _by_row(h, tables.row_token)) and torch.equal(y.double(), want)
    # d_a from S, one row for each column of x (the rest of x is 0); d_b from hidden, one row for each column of d_y
    t = torch.arange(T, device="cuda")
    first = t < min(K, N)
    at = t % min(K, N)
    one_x, one_y = torch.zeros((T, K), device="cuda"), torch.zeros((T, N), device="cuda")
    one_x[t, at], one_y[t, at] = first * (1.0 - 2 * (t % 2)), first * (1.0 - 2 * (t % 5 == 0))
    one_x, one_y = one_x.to(torch.bfloat16), one_y.to(torch.bfloat16)
    wide_b, d_y = (_large((E, N, r), g) * rank_sign).to(torch.bfloat16), _large((T, N), g).to(torch.bfloat16)
    d_y[~first] = 0
    d_x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    want, _ = _want_grads(d_x, d_y, one_x, a, wide_b, torch.zeros_like(h), ids, None)
    forms = [one_x]
    if K % 32 == 0:
        q, s = mx.quantize(one_x, 1)
        w = mx.repack(q.view(1, T, K), s.view(1, T, K // 32))
        forms += [(q, s), mx.PackedWeight(w.q, w.s, 1, T, K)]
    for form in forms:
        d_a, _ = mx.lora_backward_(None, d_y, form, a, wide_b, torch.zeros_like(hidden), tables)
        assert torch.equal(d_a.double(), want[1])
    want, _ = _want_grads(d_x, one_y, one_x, a, b, h, ids, None)
    _, d_b = mx.lora_backward_(None, one_y, one_x, a, b, hidden, tables)
    assert torch.equal(d_b.double(), want[2])
