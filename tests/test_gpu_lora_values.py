"""The low-rank adapters' operands at the ends of their range: infinite values
against finite ones, sums close to fp32's largest number, and products that
leave it.  The reference is the formula in fp64, rounded to the result's type:
finite values, infinities and NaN have to be the same (sums of whole numbers
below 2^24, or one product with a power of two: exact)."""
import pytest
import torch

from test_gpu_lora import _by_row, _gen, _ids, _whole

pytestmark = pytest.mark.gpu

INF = float("inf")
BIG = (2 - 2.0 ** -7) * 2.0 ** 127              # bf16's largest number
REST = 3 * 2.0 ** -9 * 2.0 ** 127               # BIG + REST is below fp32's largest and above what bf16 rounds to infinity


def _same(got, want):
    want = want.to(got.device).to(got.dtype)
    return torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(0, INF, -INF), want.nan_to_num(0, INF, -INF))


def _formula(x, a, b, d_y, ids, scales, h=None):
    """fp64 on the CPU: the adapters' share of y, hidden by token, the share of d_x, d_a, d_b"""
    x, a, b, d_y, ids, scales = (t.double().cpu() if t.is_floating_point() else t.cpu() for t in (x, a, b, d_y, ids, scales))
    T, (E, r, K), N = x.shape[0], a.shape, b.shape[1]
    y, d_x = torch.zeros((T, N), dtype=torch.float64), torch.zeros((T, K), dtype=torch.float64)
    hidden = torch.zeros((T, r), dtype=torch.float64)
    d_a, d_b = torch.zeros_like(a), torch.zeros_like(b)
    for e in range(E):
        t = torch.nonzero(ids == e).squeeze(1)
        if not t.numel():
            continue
        hidden[t] = x[t] @ a[e].t() if h is None else h.double().cpu()[t]
        y[t] = (scales[e] * hidden[t]) @ b[e].t()
        s = scales[e] * (d_y[t] @ b[e])
        d_x[t] = s @ a[e]
        d_a[e] = s.t() @ x[t]
        d_b[e] = d_y[t].t() @ (scales[e] * hidden[t])
    return y, hidden, d_x, d_a, d_b


def _check(mx, x, a, b, d_y, ids, scales, h=None, forms=True, sums=True):
    """Both directions, every form of x that holds it; h: hidden rows other than a's product; sums: those over rows too"""
    T, (E, r, K), N = x.shape[0], a.shape, b.shape[1]
    tables = mx.route_tables(ids.view(-1, 1), E)
    y, hidden, d_x, d_a, d_b = _formula(x, a, b, d_y, ids, scales, h)
    if h is None:
        for dtype in (torch.bfloat16, torch.float32):
            got = torch.zeros((T, N), dtype=dtype, device="cuda")
            kept = mx.lora_add_(got, x, a, b, tables, scales, keep_hidden=True)
            assert _same(got, y), dtype
            assert _same(kept, _by_row(hidden, tables.row_token.cpu()))
    inputs = [x]
    if K % 32 == 0 and forms:
        q, s = mx.quantize(x, 1)
        assert torch.equal(mx.dequantize(q, s, T, K, 1, torch.bfloat16), x)
        w = mx.repack(q.view(1, T, K), s.view(1, T, K // 32))
        inputs += [(q, s), mx.PackedWeight(w.q, w.s, 1, T, K)]
    room = _by_row(hidden.cuda(), tables.row_token).float()
    for form in inputs:
        got = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
        got_a, got_b = mx.lora_backward_(got, d_y, form, a, b, room, tables, scales)
        assert _same(got, d_x) and (not sums or (_same(got_a, d_a) and _same(got_b, d_b)))


SHAPES = [(40, 2, 8, 64, 72), (40, 2, 16, 96, 64), (150, 3, 32, 128, 136), (150, 3, 64, 64, 200), (90, 2, 128, 64, 64), (700, 1, 24, 64, 64)]


def _inputs(T, E, r, K, N, seed):
    g = _gen(seed)
    x, a, b, d_y = _whole((T, K), g, 2), _whole((E, r, K), g, 2), _whole((E, N, r), g, 2), _whole((T, N), g, 2)
    # sums that one bf16 holds, that take two (518, 525 and others, rounded up and down), and that are 0
    x[:, 0], a[:, ::2, 0] = 14, 37            # 14: MXFP8 holds it
    a[:, 3] = 0
    d_y[:, 0], b[:, 0, ::2] = 15, 35
    b[:, :, 5] = 0
    scales = 2.0 ** torch.randint(-1, 2, (E,), generator=g, device="cuda").float()
    return x, a, b, d_y, _ids(T, E, seed), scales


@pytest.mark.parametrize("T,E,r,K,N", SHAPES)
def test_infinite_weights(mx, T, E, r, K, N):
    x, a, b, d_y, ids, scales = _inputs(T, E, r, K, N, T + r)
    _check(mx, x, a, b, d_y, ids, scales)
    b[0, 7, 0], b[0, 9, 3], b[E - 1, 11, 2], b[E - 1, 13, 7] = INF, INF, -INF, -INF
    b[0, 20, 0], b[0, 20, 2] = INF, INF
    _check(mx, x, a, b, d_y, ids, scales)
    x, a, b, d_y, ids, scales = _inputs(T, E, r, K, N, T + r + 1)
    a[0, 0, 7], a[0, 5, 9], a[E - 1, 2, 11], a[E - 1, 4, 0] = INF, INF, -INF, -INF
    _check(mx, x, a, b, d_y, ids, scales)


# both products in launches of their own, the second with one step of columns and with several
MANY = [(8800, 3, 16, 64, 72), (8800, 3, 64, 64, 72), (9200, 3, 16, 64, 2056), (9200, 3, 40, 64, 2048), (4300, 2, 72, 64, 2048)]


@pytest.mark.parametrize("T,E,r,K,N", MANY)
def test_infinite_weights_of_many_rows(mx, T, E, r, K, N):
    """Sums over so many rows are not exact in fp32 and left to the other shapes"""
    x, a, b, d_y, ids, scales = _inputs(T, E, r, K, N, T + r)
    b[0, 7, 0], b[0, 9, 3], b[E - 1, 11, 2], b[E - 1, N - 1, 7] = INF, INF, -INF, -INF
    _check(mx, x, a, b, d_y, ids, scales, forms=False, sums=False)
    x, a, b, d_y, ids, scales = _inputs(T, E, r, N, K, T + r + 1)            # d_x has N columns
    a[0, 0, 7], a[0, 5, 9], a[E - 1, 2, 11], a[E - 1, 4, N - 1] = INF, INF, -INF, -INF
    _check(mx, x, a, b, d_y, ids, scales, forms=False, sums=False)


@pytest.mark.parametrize("T,E,r,K,N", SHAPES)
def test_infinite_rows(mx, T, E, r, K, N):
    x, a, b, d_y, ids, scales = _inputs(T, E, r, K, N, T + r + 2)
    ids[:] = torch.where(ids < 0, 0, ids)
    x[5, 9], x[17, 0], x[30, 3] = INF, -INF, INF
    _check(mx, x, a, b, d_y, ids, scales, forms=False)
    h = _whole((T, r), _gen(T), 300, torch.float32)
    _check(mx, x, a, b, d_y, ids, scales, h=h, forms=False)
    x, a, b, d_y, ids, scales = _inputs(T, E, r, K, N, T + r + 3)
    d_y[5, 9], d_y[17, 0], d_y[30, 3] = INF, -INF, INF
    _check(mx, x, a, b, d_y, ids, scales, h=h)
    h[4, 2], h[8, 0], h[9, 1] = INF, -INF, float("nan")
    d_y[5, 9], d_y[17, 0], d_y[30, 3] = 1, 2, 0
    _check(mx, x, a, b, d_y, ids, scales, h=h)


@pytest.mark.parametrize("T,E,r,K,N", SHAPES)
def test_sums_next_to_the_largest_number(mx, T, E, r, K, N):
    """A x and S above what bf16 rounds to infinity, times powers of two that bring them back, or past fp32's range"""
    ids = _ids(T, E, T)
    x, a = torch.zeros((T, K), device="cuda"), torch.zeros((E, r, K), device="cuda")
    b, d_y = torch.zeros((E, N, r), device="cuda"), torch.zeros((T, N), device="cuda")
    sign = torch.where(torch.arange(T, device="cuda") % 3 == 0, -1.0, 1.0)
    x[:, 0], x[:, 33] = sign * BIG, sign * REST
    a[:, 1::2, 0] = a[:, 1::2, 33] = 1
    n = torch.arange(N, device="cuda")
    b[:, n, (2 * n + 1) % r] = 2.0 ** -60
    b[:, 3, 1] = 4                                          # past fp32
    d_y[:, 0], d_y[:, 2] = sign * BIG, sign * REST
    scales = torch.ones(E, device="cuda")
    x, a, b, d_y = (t.to(torch.bfloat16) for t in (x, a, b, d_y))
    tables = mx.route_tables(ids.view(-1, 1), E)
    y, hidden, _, _, _ = _formula(x, a, b, d_y, ids, scales)
    assert float(hidden.abs().max()) == BIG + REST
    for dtype in (torch.bfloat16, torch.float32):
        got = torch.zeros((T, N), dtype=dtype, device="cuda")
        kept = mx.lora_add_(got, x, a, b, tables, scales, keep_hidden=True)
        assert _same(kept, _by_row(hidden, tables.row_token.cpu())) and _same(got, y)
    # S = d_y b: one row of d_x each, one row for each entry of d_a
    b, x, a = torch.zeros_like(b), torch.zeros_like(x), torch.zeros_like(a)
    b[:, 0, 2], b[:, 2, 2] = 1, 1
    a[:, 2, 5], a[:, 2, 6] = 2.0 ** -60, 4
    t = torch.arange(T, device="cuda")
    x[t, t % K] = torch.where(t < K, 2.0 ** -30, 0.0).to(torch.bfloat16)
    h = torch.zeros((T, r), device="cuda")
    h[0] = (2 - 2.0 ** -23) * 2.0 ** 127
    h[7, 3] = -h[0, 0]
    d_y[:, 10:] = 0
    d_y[0, 10], d_y[7, 11] = 2.0 ** -30, 2.0 ** -90
    d_y[1:, :3] = torch.where(torch.arange(T - 1, device="cuda").unsqueeze(1) < K - 1, d_y[1:, :3].float(), 0.0).to(torch.bfloat16)
    ids[0] = ids[7] = 0
    _check(mx, x, a, b, d_y, ids, scales, h=h)


def test_products_past_the_range(mx):
    """The parts of a sum leave fp32 with opposite signs; the product is an infinity all the same"""
    for T, E, r, K, N in SHAPES:
        ids = _ids(T, E, T, none=False)
        x, a = torch.zeros((T, K), device="cuda"), torch.zeros((E, r, K), device="cuda")
        x[:, 0], x[:, 1] = 2.0 ** 101, -2.0 ** 91           # 2^101 - 2^91: in parts 2^101 and -2^91
        x[1::2] *= -1
        a[:, :, 0] = a[:, :, 1] = 1
        b, d_y = torch.zeros((E, N, r), device="cuda"), torch.zeros((T, N), device="cuda")
        b[:, torch.arange(N), torch.arange(N) % r] = 2.0 ** 40
        d_y[:, 0], d_y[:, 1] = 2.0 ** 61, -2.0 ** 51        # S = 2^40 (2^61, -2^51) at ranks 0 and 1
        d_y[1::2] *= -1
        x, a, b, d_y = (t.to(torch.bfloat16) for t in (x, a, b, d_y))
        b[:, 0, 2], b[:, 1, 2] = 2.0 ** 40, 2.0 ** 40       # at rank 2: 2^101 - 2^91
        _check(mx, x, a, b, d_y, ids, torch.ones(E, device="cuda"), forms=False)
