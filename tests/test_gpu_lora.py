"""The low-rank adapters on the GPU: products and gradients against fp64.

Small whole numbers make every step exact (sums below 2^24, hidden values below
2^16, which two bf16 numbers hold), so those tests ask for equality.  With real
values the bound of a sum of n fp32 products is n 2^-23 of the sum of their
sizes, in any order and if each addition truncates; a value that enters a
product as two bf16 numbers loses 2^-16 of it (half a step of bf16, 2^-8,
twice); the result is rounded once, half a step of its type.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
SUM, SPLIT = 2.0 ** -23, 2.0 ** -16


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ids(T, E, seed, none=True):
    """Adapters in runs; some rows without one, some adapters without rows."""
    g = _gen(seed)
    ids = torch.randint(-1 if none else 0, E, (T,), generator=g, device="cuda")
    ids = torch.where(torch.rand(T, generator=g, device="cuda") < 0.7, ids[torch.arange(T, device="cuda") // 5 * 5], ids)
    return ids.to(torch.int32)


def _whole(shape, g, most, dtype=torch.bfloat16):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(dtype)


def _want(y, x, a, b, ids, scales):
    """fp64: y, hidden by token, and the sums of the terms' sizes"""
    out, size = y.double().clone(), torch.zeros(y.shape, dtype=torch.float64, device="cuda")
    h = torch.zeros((x.shape[0], a.shape[1]), dtype=torch.float64, device="cuda")
    hsize = h.clone()
    for e in range(a.shape[0]):
        t = torch.nonzero(ids == e).squeeze(1)
        if not t.numel():
            continue
        s = scales[e].double() if scales is not None else 1.0
        h[t] = x[t].double() @ a[e].double().t().contiguous()
        hsize[t] = x[t].double().abs() @ a[e].double().abs().t().contiguous()
        bt = b[e].double().t().contiguous()
        out[t] += s * (h[t] @ bt)
        K, r = a.shape[2], a.shape[1]
        size[t] = abs(s) * ((hsize[t] * K * SUM + h[t].abs() * (SPLIT + 2.0 ** -23)) @ bt.abs() + 2 * (r + 8) * SUM * (h[t].abs() @ bt.abs()))
    return out, h, size, hsize * a.shape[2] * SUM


def _by_row(h, row_token):
    return torch.where(row_token.unsqueeze(1) >= 0, h[row_token.clamp_min(0)], torch.zeros_like(h[:1]))


SHAPES = [  # T, E, r, K, N
    (1, 1, 8, 64, 72), (1, 8, 16, 4096, 1536), (5, 3, 24, 136, 264), (33, 2, 32, 512, 256), (64, 70, 8, 1000, 40),
    (127, 5, 40, 648, 320), (250, 64, 16, 2048, 1288), (300, 1, 64, 1024, 512), (513, 4, 128, 256, 640), (2100, 9, 48, 384, 2000),
    (700, 200, 16, 96, 96), (40, 1024, 8, 64, 64)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,r,K,N", SHAPES)
def test_add_exact(mx, T, E, r, K, N, dtype):
    g = _gen(T + r)
    ids = _ids(T, E, T)
    x, a, b = _whole((T, K), g, 1), _whole((E, r, K), g, 1), _whole((E, N, r), g, 1)
    scales = 2.0 ** torch.randint(-1, 2, (E,), generator=g, device="cuda").float()
    y = _whole((T, N), g, 4, dtype)
    want, h, _, _ = _want(y, x, a, b, ids, scales)
    tables = mx.route_tables(ids.view(-1, 1), E)
    hidden = mx.lora_add_(y, x, a, b, tables, scales, keep_hidden=True)
    assert torch.equal(hidden.double(), _by_row(h, tables.row_token))
    assert torch.equal(y, want.to(dtype))


@pytest.mark.parametrize("T,E,r,K,N", SHAPES)
def test_add(mx, T, E, r, K, N):
    g = _gen(T + r + 1)
    ids = _ids(T, E, T + 1)
    x = torch.randn((T, K), generator=g, device="cuda").to(torch.bfloat16)
    a = (torch.randn((E, r, K), generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16)
    b = torch.randn((E, N, r), generator=g, device="cuda").to(torch.bfloat16)
    scales = torch.rand(E, generator=g, device="cuda") + 0.25
    tables = mx.route_tables(ids.view(-1, 1), E)
    for dtype in (torch.bfloat16, torch.float32):
        for s in (scales, None):
            y = torch.randn((T, N), generator=g, device="cuda").to(dtype)
            want, h, size, hsize = _want(y, x, a, b, ids, s)
            hidden = mx.lora_add_(y, x, a, b, tables, s, keep_hidden=True)
            assert bool(((hidden.double() - _by_row(h, tables.row_token)).abs() <= _by_row(hsize, tables.row_token)).all())
            assert bool(((y.double() - want).abs() <= size * 1.01 + HALF[dtype] * (want.abs() + size) * 1.01).all())


def _want_grads(d_x, d_y, x, a, b, h, ids, scales):
    d_x = d_x.double().clone()
    d_a, d_b = torch.zeros(a.shape, dtype=torch.float64, device="cuda"), torch.zeros(b.shape, dtype=torch.float64, device="cuda")
    sizes = [torch.zeros_like(t) for t in (d_x, d_a, d_b)]
    N, r = b.shape[1:]
    for e in range(a.shape[0]):
        t = torch.nonzero(ids == e).squeeze(1)
        if not t.numel():
            continue
        s = scales[e].double() if scales is not None else 1.0
        dy, ae, be, n = d_y[t].double(), a[e].double(), b[e].double(), t.numel() + 8
        S = s * (dy @ be)
        off = abs(s) * (dy.abs() @ be.abs()) * (N * SUM) + S.abs() * (SPLIT + 2.0 ** -23)      # of S as an operand
        d_x[t] += S @ ae
        sizes[0][t] = off @ ae.abs() + 2 * (r + 8) * SUM * (S.abs() @ ae.abs())
        St, xt = S.t().contiguous(), x[t].double()
        d_a[e] = St @ xt
        sizes[1][e] = off.t().contiguous() @ xt.abs() + 2 * n * SUM * (St.abs() @ xt.abs())
        dyt = dy.t().contiguous() * s
        d_b[e] = dyt @ h[t].double()
        sizes[2][e] = (2 * n * SUM + SPLIT + 2.0 ** -23) * (dyt.abs() @ h[t].double().abs())
    return (d_x, d_a, d_b), sizes


def _forms(mx, x):
    """x in every form that holds it exactly"""
    T, K = x.shape
    yield x
    if K % 32 == 0:
        q, s = mx.quantize(x, 1)
        if torch.equal(mx.dequantize(q, s, T, K, 1, torch.bfloat16), x):
            yield q, s
            w = mx.repack(q.view(1, T, K), s.view(1, T, K // 32))
            yield mx.PackedWeight(w.q, w.s, 1, T, K)


@pytest.mark.parametrize("T,E,r,K,N", SHAPES)
def test_gradients_exact(mx, T, E, r, K, N):
    g = _gen(T + r + 2)
    ids = _ids(T, E, T + 2)
    tables = mx.route_tables(ids.view(-1, 1), E)
    x, a, b, d_y = _whole((T, K), g, 2), _whole((E, r, K), g, 1), _whole((E, N, r), g, 1), _whole((T, N), g, 1)
    scales = 2.0 ** torch.randint(-1, 2, (E,), generator=g, device="cuda").float()
    h = _whole((T, r), g, 100, torch.float32)
    hidden = _by_row(h, tables.row_token)
    d_x = _whole((T, K), g, 4)
    want, _ = _want_grads(d_x, d_y, x, a, b, h, ids, scales)
    forms = 0
    for form in _forms(mx, x):
        got_x = d_x.clone()
        d_a, d_b = mx.lora_backward_(got_x, d_y, form, a, b, hidden, tables, scales)
        assert torch.equal(d_a.double(), want[1]) and torch.equal(d_b.double(), want[2])
        assert torch.equal(got_x, want[0].to(torch.bfloat16))
        alone = mx.lora_backward_(None, d_y, form, a, b, hidden, tables, scales)
        assert torch.equal(alone[0], d_a) and torch.equal(alone[1], d_b)
        forms += 1
    assert forms == (3 if K % 32 == 0 else 1)


@pytest.mark.parametrize("T,E,r,K,N", SHAPES)
def test_gradients(mx, T, E, r, K, N):
    g = _gen(T + r + 3)
    ids = _ids(T, E, T + 3)
    tables = mx.route_tables(ids.view(-1, 1), E)
    x = (torch.randn((T, K), generator=g, device="cuda") * 2.0 ** torch.randint(-6, 7, (T, 1), generator=g, device="cuda")).to(torch.bfloat16)
    a = (torch.randn((E, r, K), generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16)
    b = torch.randn((E, N, r), generator=g, device="cuda").to(torch.bfloat16)
    d_y = torch.randn((T, N), generator=g, device="cuda").to(torch.bfloat16)
    h = torch.randn((T, r), generator=g, device="cuda")
    d_x = torch.randn((T, K), generator=g, device="cuda").to(torch.bfloat16)
    scales = torch.rand(E, generator=g, device="cuda") + 0.25
    forms = [(x, x)]
    if K % 32 == 0:
        q, s = mx.quantize(x, 1)
        kept = mx.dequantize(q, s, T, K, 1, torch.float32)
        w = mx.repack(q.view(1, T, K), s.view(1, T, K // 32))
        forms += [((q, s), kept), (mx.PackedWeight(w.q, w.s, 1, T, K), kept)]
    for form, value in forms:
        for sc in (scales, None):
            want, size = _want_grads(d_x, d_y, value, a, b, h, ids, sc)
            got_x = d_x.clone()
            got = (got_x,) + mx.lora_backward_(got_x, d_y, form, a, b, _by_row(h, tables.row_token), tables, sc)
            for u, v, z in zip(got, want, size):
                assert bool(((u.double() - v).abs() <= z * 1.01 + HALF[u.dtype] * (v.abs() + z) * 1.01).all())


def test_gradients_are_the_differences_of_the_product(mx):
    """The product is linear in b and in a; with whole numbers its differences are exact."""
    T, E, r, K, N = 70, 2, 8, 64, 40
    g = _gen(11)
    ids = _ids(T, E, 4)
    tables = mx.route_tables(ids.view(-1, 1), E)
    x, a, b = _whole((T, K), g, 2), _whole((E, r, K), g, 2), _whole((E, N, r), g, 2)
    c = _whole((T, N), g, 2)
    scales = torch.tensor([0.5, 2.0], device="cuda")

    def loss(x, a, b):
        y = torch.zeros((T, N), device="cuda")
        hidden = mx.lora_add_(y, x, a, b, tables, scales, keep_hidden=True)
        return (y.double() * c.double()).sum().item(), hidden
    base, hidden = loss(x, a, b)
    d_x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    d_a, d_b = mx.lora_backward_(d_x, c, x, a, b, hidden, tables, scales)
    for e, j, k in ((0, 0, 0), (1, 7, 63), (0, 3, 17)):
        up = a.clone()
        up[e, j, k] += 1
        assert loss(x, up, b)[0] - base == d_a[e, j, k].item()
    for e, n, j in ((0, 0, 0), (1, 39, 7), (1, 11, 2)):
        up = b.clone()
        up[e, n, j] += 1
        assert loss(x, a, up)[0] - base == d_b[e, n, j].item()
    for t, k in ((0, 0), (69, 63), (33, 5)):
        up = x.clone()
        up[t, k] += 1
        assert torch.tensor(loss(up, a, b)[0] - base).to(torch.bfloat16).item() == d_x[t, k].item()


def test_rows_without_an_adapter_are_left_alone(mx):
    """Neither read nor written, whatever they hold; strided rows' gaps too."""
    T, E, r, K, N = 90, 3, 16, 96, 88
    g = _gen(5)
    ids = _ids(T, E, 9)
    ids[::7] = -1
    ids[3], ids[4] = E, 1 << 30
    tables = mx.route_tables(ids.view(-1, 1), E)
    none = (ids < 0) | (ids >= E)
    x_wide, y_wide = _whole((T, K + 24), g, 1), _whole((T, N + 16), g, 4, torch.float32)
    x_wide[none], y_wide[none] = float("nan"), float("nan")
    x, y = x_wide[:, 8:8 + K], y_wide[:, 8:8 + N]
    a, b = _whole((E, r, K), g, 1), _whole((E, N, r), g, 1)
    want, h, _, _ = _want(y.contiguous(), torch.where(none.unsqueeze(1), 0, x), a, b, ids, None)
    before = y_wide.clone()
    hidden = mx.lora_add_(y, x, a, b, tables, keep_hidden=True)
    assert torch.equal(y[~none], want[~none].float())
    changed = before.clone()
    changed[:, 8:8 + N][~none] = want[~none].float()
    assert torch.equal(y_wide.view(torch.int32), changed.view(torch.int32))
    assert torch.equal(hidden.double(), _by_row(h, tables.row_token))
    d_y, d_x = _whole((T, N + 8), g, 1), _whole((T, K + 8), g, 4)
    d_y[none], d_x[none] = float("inf"), float("nan")
    keep = d_x.clone()
    want, _ = _want_grads(d_x[:, :K], torch.where(none.unsqueeze(1), 0, d_y[:, :N]), torch.where(none.unsqueeze(1), 0, x), a, b, h, ids, None)
    d_a, d_b = mx.lora_backward_(d_x[:, :K], d_y[:, :N], x, a, b, hidden, tables)
    assert torch.equal(d_a.double(), want[1]) and torch.equal(d_b.double(), want[2])
    keep[:, :K][~none] = want[0][~none].to(torch.bfloat16)
    assert torch.equal(d_x.view(torch.int16), keep.view(torch.int16))


def test_nan_and_inf_stay_in_their_rows(mx):
    T, E, r, K, N = 64, 2, 16, 64, 64
    g = _gen(6)
    ids = _ids(T, E, 1, none=False)
    tables = mx.route_tables(ids.view(-1, 1), E)
    x, a, b = _whole((T, K), g, 1), _whole((E, r, K), g, 1), _whole((E, N, r), g, 1)
    a[:, :, 3] = 1
    clean = torch.zeros((T, N), device="cuda")
    mx.lora_add_(clean, x, a, b, tables)
    x[10, 3], x[20, 3] = float("nan"), float("inf")
    y = torch.zeros((T, N), device="cuda")
    hidden = mx.lora_add_(y, x, a, b, tables, keep_hidden=True)
    rows = torch.ones(T, dtype=torch.bool, device="cuda")
    rows[10] = rows[20] = False
    assert torch.equal(y[rows], clean[rows])
    assert bool(y[10].isnan().all()) and not bool(torch.isfinite(y[20]).any())
    at = torch.nonzero(tables.row_token == 20).item()
    assert bool((hidden[at] == float("inf")).all())


def test_tables_without_rows_and_tokens(mx):
    E, r, K, N = 3, 8, 64, 64
    a = torch.ones((E, r, K), dtype=torch.bfloat16, device="cuda")
    b = torch.ones((E, N, r), dtype=torch.bfloat16, device="cuda")
    x, y = torch.ones((6, K), dtype=torch.bfloat16, device="cuda"), torch.ones((6, N), device="cuda")
    ids = torch.full((6, 1), -1, dtype=torch.int32, device="cuda")
    tables = mx.route_tables(ids, E)
    hidden = mx.lora_add_(y, x, a, b, tables, keep_hidden=True)
    assert bool((y == 1).all()) and bool((hidden == 0).all()) and hidden.shape[0] == tables.row_token.numel() > 0
    d_a, d_b = mx.lora_backward_(None, y.to(torch.bfloat16), x, a, b, hidden, tables)
    assert bool((d_a == 0).all()) and bool((d_b == 0).all())
    # no tokens, with and without rows in the tables
    for rows in (0, 64):
        tables = mx.route_tables(ids[:0], E, rows=rows)
        hidden = mx.lora_add_(y[:0], x[:0], a, b, tables, keep_hidden=True)
        assert hidden.shape == (rows, r) and bool((hidden == 0).all())
        d_a, d_b = mx.lora_backward_(x[:0].clone(), y[:0].to(torch.bfloat16), x[:0], a, b, hidden, tables)
        assert bool((d_a == 0).all()) and bool((d_b == 0).all())


def test_one_adapter_with_nearly_all_rows(mx):
    """Skewed groups: one adapter's sums come from many chunks, the others' from one or none."""
    T, E, r, K, N = 6000, 40, 16, 128, 136
    g = _gen(8)
    ids = torch.zeros(T, dtype=torch.int32, device="cuda") + 7
    ids[:90] = torch.randint(0, 20, (90,), generator=g, device="cuda").to(torch.int32)
    ids[5000:5600] = 33
    tables = mx.route_tables(ids.view(-1, 1), E)
    x, a, b, d_y = _whole((T, K), g, 2), _whole((E, r, K), g, 1), _whole((E, N, r), g, 1), _whole((T, N), g, 1)
    h = _whole((T, r), g, 60, torch.float32)
    d_x = _whole((T, K), g, 4)
    want, _ = _want_grads(d_x, d_y, x, a, b, h, ids, None)
    d_a, d_b = mx.lora_backward_(d_x, d_y, x, a, b, _by_row(h, tables.row_token), tables)
    assert torch.equal(d_a.double(), want[1]) and torch.equal(d_b.double(), want[2])
    assert torch.equal(d_x, want[0].to(torch.bfloat16))


def test_same_bits_every_time(mx):
    T, E, r, K, N = 1500, 6, 32, 512, 520
    g = _gen(9)
    ids = _ids(T, E, 3)
    tables = mx.route_tables(ids.view(-1, 1), E)
    x, d_y = (torch.randn((T, n), generator=g, device="cuda").to(torch.bfloat16) for n in (K, N))
    a, b = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16) for s in ((E, r, K), (E, N, r)))
    runs = []
    for _ in range(3):
        y, d_x = torch.zeros((T, N), device="cuda"), torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
        hidden = mx.lora_add_(y, x, a, b, tables, keep_hidden=True)
        runs.append((y, hidden, d_x) + mx.lora_backward_(d_x, d_y, x, a, b, hidden, tables))
    for other in runs[1:]:
        assert all(torch.equal(u, v) for u, v in zip(runs[0], other))


def test_streams_and_graphs(mx):
    """Two captured graphs and eager calls between their replays; each call has a workspace of its own."""
    T, E, r, K, N = 200, 4, 16, 256, 264
    g = _gen(10)
    a, b = _whole((E, r, K), g, 1), _whole((E, N, r), g, 1)
    data = []
    for s in range(2):
        ids = _ids(T, E, 20 + s)
        data.append((ids, _whole((T, K), g, 1), _whole((T, N), g, 4), _whole((T, N), g, 1), _whole((T, K), g, 2)))

    def step(ids, x, y, d_y, d_x):
        tables = mx.route_tables(ids.view(-1, 1), E)
        hidden = mx.lora_add_(y, x, a, b, tables, keep_hidden=True)
        return (y, hidden, d_x) + mx.lora_backward_(d_x, d_y, x, a, b, hidden, tables)
    want = [step(i, x, y.clone(), dy, dx.clone()) for i, x, y, dy, dx in data]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(data[1][0], data[1][1], data[1][2].clone(), data[1][3], data[1][4].clone())
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want[1]))
    graphs = []
    for k in range(2):
        inputs = [t.clone() for t in data[k]]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(*inputs)
        graphs.append((graph, inputs, out))
    for k, n in ((0, 0), (1, 1), (0, 1), (1, 0), (0, 0)):
        graph, inputs, out = graphs[k]
        for t, v in zip(inputs, data[n]):
            t.copy_(v)
        graph.replay()
        step(data[n][0], data[n][1], data[n][2].clone(), data[n][3], data[n][4].clone())
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(out, want[n])), (k, n)


def test_rows_2_31_elements_apart(mx):
    T, E, r, K, N = 3, 2, 8, 64, 64
    g = _gen(12)
    ids = torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda")
    tables = mx.route_tables(ids.view(-1, 1), E)
    ld = (1 << 30) + 8
    room = torch.zeros(2 * ld + 64, dtype=torch.bfloat16, device="cuda")
    far = room.as_strided((T, 64), (ld, 1))
    a, b, x = _whole((E, r, K), g, 1), _whole((E, N, r), g, 1), _whole((T, K), g, 1)
    y = _whole((T, N), g, 2, torch.float32)
    want, h, _, _ = _want(y, x, a, b, ids, None)
    far.copy_(x)
    mx.lora_add_(y, far, a, b, tables)
    assert torch.equal(y, want.float())
    far.copy_(y.to(torch.bfloat16))
    mx.lora_add_(far, x, a, b, tables)
    twice = _want(y.to(torch.bfloat16), x, a, b, ids, None)[0]
    assert torch.equal(far, twice.to(torch.bfloat16))


def test_malformed_tables_stay_inside(mx):
    """Offsets in any order and tokens of any value: whatever comes out, nothing outside the outputs is written and the
    next call is right.  (The addresses themselves are followed on the CPU in test_lora_tables.py.)"""
    T, E, r, K, N = 100, 5, 8, 64, 64
    g = _gen(13)
    x, a, b, d_y = _whole((T, K), g, 1), _whole((E, r, K), g, 1), _whole((E, N, r), g, 1), _whole((T, N), g, 1)
    good = mx.route_tables(_ids(T, E, 30).view(-1, 1), E)
    rows = good.row_token.numel()
    y0 = torch.zeros((T, N), device="cuda")
    mx.lora_add_(y0, x, a, b, good)
    for offsets in ([0, rows, 0, rows, 0, rows], [-64, -32, 7, 45, 1 << 30, 3], [rows] * 6, [96, 64, 32, 0, 160, 32]):
        bad = mx.RouteTables(torch.tensor(offsets, dtype=torch.int32, device="cuda"), good.counts,
                             torch.randint(-T, 2 * T, (rows,), generator=g, device="cuda"), good.pair_row, 32)
        room = torch.full((T + 2, N), 7.0, device="cuda")
        hidden = mx.lora_add_(room[1:-1], x, a, b, bad, keep_hidden=True)
        assert bool((room[0] == 7).all()) and bool((room[-1] == 7).all())
        mx.lora_backward_(None, d_y, x, a, b, hidden, bad)
    y = torch.zeros((T, N), device="cuda")
    mx.lora_add_(y, x, a, b, good)
    assert torch.equal(y, y0)


# Sizes on both sides of the rule that takes both products in one launch (rank up to 64): below it by the length of a
# block's rows, by blocks for every second CU, and above it by more blocks than there are CUs.
RULE = [(1, 1, 16, 6128, 200), (1, 1, 16, 6144, 200), (512, 8, 16, 4096, 1032), (90, 3, 64, 2056, 328), (90, 3, 32, 4104, 72),
        (4200, 3, 64, 264, 584), (8600, 9, 40, 72, 136), (8900, 5, 16, 136, 264), (9100, 2, 64, 200, 456), (9100, 2, 32, 520, 64),
        (4200, 3, 16, 16392, 72)]


@pytest.mark.parametrize("T,E,r,K,N", RULE)
def test_one_launch_or_two(mx, T, E, r, K, N):
    for dtype in (torch.bfloat16, torch.float32):
        test_add_exact(mx, T, E, r, K, N, dtype)
    test_add(mx, T, E, r, K, N)
    test_gradients_exact(mx, T, E, r, K, N)
    test_gradients_exact(mx, T, E, r, N, K)
    test_gradients(mx, T, E, r, K, N)
