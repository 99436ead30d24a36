"""Expert routing, its gradient and the row tables against plain fp64 forms."""
import numpy as np
import pytest
import torch

import workloads as wl

pytestmark = pytest.mark.gpu

HALF32 = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
# scores: exponential 4 half steps, at most 22 additions in the sum, division, product with 1/sum;
# renormalizing: at most 6 more additions, a division; scale
WEIGHT_TOL = 48 * HALF32


def _scores(x, score):
    x = x.astype(np.float64)
    if score == "sigmoid":
        return 1.0 / (1.0 + np.exp(-x))
    e = np.exp(x - x.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def _route(x, k, score="softmax", bias=None, groups=1, groups_kept=1, group_top=1, renormalize=True, scale=1.0):
    s = _scores(x, score)
    c = s if bias is None else s + bias.astype(np.float64)
    T, E = c.shape
    if groups > 1:
        g = -np.sort(-c.reshape(T, groups, -1), axis=2)[:, :, :group_top].sum(2)
        order = np.argsort(-g, axis=1, kind="stable")
        shut = np.ones((T, groups), bool)
        np.put_along_axis(shut, order[:, :groups_kept], False, 1)
        c = np.where(np.repeat(shut, E // groups, 1), -np.inf, c)
    ids = np.argsort(-c, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(s, ids, 1)
    if renormalize:
        w = w / w.sum(1, keepdims=True)
    return ids, w * scale


def _logits(T, E, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn((T, E), generator=g, device="cuda") * 1.5).to(dtype)


def _check(mx, x, k, **kw):
    bias = kw.pop("bias", None)
    ids, w = mx.route(x, k, bias=bias, **kw)
    want_ids, want_w = _route(x.float().cpu().numpy(), k, bias=None if bias is None else bias.cpu().numpy(), **kw)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    got = w.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - want_w) <= WEIGHT_TOL * np.abs(want_w)), np.abs(got / want_w - 1).max()
    return ids, w


CASES = [
    (1, 1, 1, torch.float32, {}),
    (3, 8, 2, torch.bfloat16, {}),
    (1, 128, 8, torch.float32, {}),
    (65, 128, 8, torch.bfloat16, dict(renormalize=False)),
    (100, 37, 5, torch.float32, dict(score="sigmoid", scale=2.5)),
    (17, 512, 32, torch.float32, dict(score="sigmoid", bias=True)),
    (33, 511, 15, torch.bfloat16, dict(bias=True)),
    (64, 300, 16, torch.float32, dict(bias=True, renormalize=False)),
    (257, 256, 8, torch.float32, dict(score="sigmoid", bias=True, groups=8, groups_kept=4, group_top=2, scale=2.5)),
    (129, 256, 8, torch.bfloat16, dict(groups=8, groups_kept=3, group_top=2)),
    (70, 185, 9, torch.float32, dict(groups=5, groups_kept=2)),
    (70, 510, 10, torch.bfloat16, dict(groups=3, groups_kept=1, group_top=2, score="sigmoid")),
    (41, 128, 6, torch.float32, dict(groups=64, groups_kept=3, group_top=2, bias=True)),
    (41, 64, 6, torch.bfloat16, dict(groups=64, groups_kept=7, bias=True)),
    (41, 60, 6, torch.bfloat16, dict(groups=4, groups_kept=4, group_top=2)),
    (41, 60, 30, torch.float32, dict(groups=4, groups_kept=2, score="sigmoid")),
]


@pytest.mark.parametrize("T,E,k,dtype,kw", CASES)
def test_route(mx, T, E, k, dtype, kw):
    kw = dict(kw)
    if kw.get("bias"):
        g = torch.Generator(device="cuda")
        g.manual_seed(T)
        kw["bias"] = torch.randn(E, generator=g, device="cuda") * 0.05
    _check(mx, _logits(T, E, dtype, 7 + T), k, **kw)


def test_route_ties_and_close_scores(mx):
    # all logits equal: lowest indices, lowest groups
    x = torch.full((5, 96), 0.25, device="cuda")
    for kw in ({}, dict(score="sigmoid"), dict(groups=8, groups_kept=2, group_top=2), dict(groups=8, groups_kept=2),
               dict(score="sigmoid", bias=torch.zeros(96, device="cuda"))):
        _check(mx, x, 7, **kw)
        _check(mx, x.bfloat16(), 7, **kw)
    # neighbouring fp32 logits: the scores differ by less than fp32 holds
    base = torch.full((64, 128), 0.7, device="cuda")
    step = torch.randint(0, 40, (64, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    x = (base.view(torch.int32) + step.int()).view(torch.float32)
    bias = torch.full((128,), 0.5, device="cuda")
    for kw in ({}, dict(score="sigmoid"), dict(bias=bias), dict(score="sigmoid", bias=bias),
               dict(score="sigmoid", bias=bias, groups=4, groups_kept=2, group_top=2)):
        _check(mx, x, 8, **kw)


def test_route_masked_and_far_logits(mx):
    x = _logits(40, 64, torch.float32, 5)
    x[:, 10:] = -float("inf")
    _check(mx, x, 8, score="softmax")
    _check(mx, x, 8, score="sigmoid", bias=torch.linspace(-0.1, 0.1, 64, device="cuda"))
    ids, w = mx.route(x, 12, renormalize=False)               # more choices than experts left
    assert torch.equal(ids[:, 10:], torch.tensor([[10, 11]] * 40, dtype=torch.int32, device="cuda"))
    assert torch.all(w[:, 10:] == 0)
    low = torch.finfo(torch.float32).min
    x = torch.full((3, 64), low, device="cuda")
    x[1, 5], x[2, 5] = 1.0, -low
    ids, w = mx.route(x, 2)
    assert ids[:, 0].tolist() == [0, 5, 5] and ids[:, 1].tolist() == [1, 0, 0]
    assert torch.equal(w, torch.tensor([[0.5, 0.5], [1, 0], [1, 0]], device="cuda"))


def test_route_empty_and_nan_rows(mx):
    x = _logits(6, 128, torch.float32, 9)
    clean_ids, clean_w = mx.route(x, 8, groups=8, groups_kept=4, group_top=2)
    x[1] = -float("inf")
    x[3, 77] = float("nan")
    x[4] = float("nan")
    ids, w = mx.route(x, 8, groups=8, groups_kept=4, group_top=2)
    for r in (0, 2, 5):                                       # neighbours are untouched
        assert torch.equal(ids[r], clean_ids[r]) and torch.equal(w[r], clean_w[r])
    for r in (1, 3, 4):
        assert torch.isnan(w[r]).all()
    for row in ids.tolist():
        assert len(set(row)) == 8 and min(row) >= 0 and max(row) < 128


def test_route_strides_streams_and_no_tokens(mx):
    wide = _logits(50, 200, torch.bfloat16, 11)
    x = wide[:, 3:131]                                        # rows start at odd elements
    ids, w = _check(mx, x, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ids2, w2 = mx.route(x, 8)
    s.synchronize()
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    ids, w = mx.route(wide[:0], 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    assert mx.route_backward(wide[:0], ids, w).shape == (0, 200)


# ------------------------------------------------------------------ gradient

def _route_grad(x, ids, dw, score, renorm, scale):
    """fp64 formula and the size of what is added up in each element."""
    s = _scores(x, score)
    rows = np.arange(x.shape[0])[:, None]
    a = s[rows, ids]
    g = dw.astype(np.float64) * scale
    size = np.abs(g)
    if renorm:
        A = a.sum(1, keepdims=True)
        size = size / A + (np.abs(g) * a).sum(1, keepdims=True) / A ** 2
        g = (g - (g * a).sum(1, keepdims=True) / A) / A
    full, bound = np.zeros_like(s), np.zeros_like(s)
    full[rows, ids], bound[rows, ids] = g, size
    if score == "sigmoid":
        return full * s * (1 - s), bound * s
    return s * (full - (g * a).sum(1, keepdims=True)), s * (bound + (size * a).sum(1, keepdims=True))


GRADS = [(1, 8, 1, torch.float32, "softmax", True), (100, 128, 8, torch.bfloat16, "softmax", False),
         (33, 37, 5, torch.float32, "sigmoid", True), (20, 512, 32, torch.float32, "softmax", True),
         (20, 511, 10, torch.bfloat16, "sigmoid", False), (9, 300, 20, torch.float32, "softmax", False)]


@pytest.mark.parametrize("T,E,k,dtype,score,renorm", GRADS)
def test_route_backward(mx, T, E, k, dtype, score, renorm):
    x = _logits(T, E + 5, dtype, 21)[:, 2:2 + E]
    ids, w = mx.route(x, k, score=score, renormalize=renorm, scale=2.5)
    dw = torch.randn((T, k), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    d = mx.route_backward(x, ids, dw, score=score, renormalize=renorm, scale=2.5)
    want, size = _route_grad(x.float().cpu().numpy(), ids.cpu().numpy(), dw.cpu().numpy(), score, renorm, 2.5)
    err = np.abs(d.double().cpu().numpy() - want)
    assert d.dtype == dtype and np.all(err <= 2 * WEIGHT_TOL * size + HALF[dtype] * np.abs(want) + 1e-37), err.max()


def test_route_backward_differences(mx):
    # sum(w * c) of the fp64 forward, central differences at every logit
    x = _logits(4, 24, torch.float32, 31)
    c = torch.randn((4, 6), device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    for score, renorm in (("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)):
        ids, _ = mx.route(x, 6, score=score, renormalize=renorm)
        d = mx.route_backward(x, ids, c, score=score, renormalize=renorm).double().cpu().numpy()
        x0, i0, c0 = x.double().cpu().numpy(), ids.cpu().numpy(), c.double().cpu().numpy()

        def f(z):
            w = np.take_along_axis(_scores(z, score), i0, 1)
            return (c0 * (w / w.sum(1, keepdims=True) if renorm else w)).sum(1)
        h = 1e-5
        for e in range(24):
            z1, z2 = x0.copy(), x0.copy()
            z1[:, e] += h
            z2[:, e] -= h
            # fp64 differences: h^2 / 6 of the third derivative (below 10 here) and 2^-52 / h of rounding
            np.testing.assert_allclose(d[:, e], (f(z1) - f(z2)) / (2 * h), rtol=0, atol=2e-6)


def test_route_backward_ignores_ids_out_of_range(mx):
    x = _logits(5, 16, torch.float32, 41)
    ids, _ = mx.route(x, 3, renormalize=False)
    dw = torch.ones((5, 3), device="cuda")
    dw0 = dw.clone()
    dw0[:, 1] = 0
    bad = ids.clone()
    bad[:, 1] = torch.tensor([-1, 16, 1 << 30, -(1 << 31), 99], device="cuda", dtype=torch.int32)
    assert torch.equal(mx.route_backward(x, bad, dw, renormalize=False), mx.route_backward(x, ids, dw0, renormalize=False))


# ------------------------------------------------------------------ tables

def _tables(ids, E, pad, rows):
    T, k = ids.shape
    counts = np.zeros(E, np.int64)
    members = [[] for _ in range(E)]
    for q, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < E:
            members[e].append(q)
    off, tok, pr = np.zeros(E + 1, np.int64), np.full(rows, -1, np.int64), np.full(T * k, -1, np.int64)
    for e in range(E):
        n = len(members[e])
        counts[e], off[e + 1] = n, off[e] + (n + pad - 1) // pad * pad
        q = np.array(members[e], np.int64)
        pr[q] = off[e] + np.arange(n)
        tok[off[e]:off[e] + n] = q // k
    return off, counts, tok, pr.reshape(T, k)


@pytest.mark.parametrize("T,k,E,pad", [(1, 1, 1, 32), (1, 8, 128, 32), (32, 8, 128, 32), (7, 3, 1024, 1),
                                       (171, 3, 5, 128), (129, 8, 512, 32), (1500, 7, 61, 32), (16384, 8, 256, 32),
                                       (9000, 10, 1024, 128), (70001, 1, 2, 1)])
def test_route_tables(mx, T, k, E, pad):
    rng = np.random.default_rng(T)
    if k <= E:
        ids = wl.zipf_topk_routing(rng, T, E, k)
    else:
        ids = rng.integers(0, E, (T, k)).astype(np.int32)
    t = mx.route_tables(torch.from_numpy(ids).cuda(), E, pad)
    rows = mx.route_rows(T * k, E, pad)
    assert t.row_token.numel() == rows
    for got, want in zip((t.offsets, t.counts, t.row_token, t.pair_row), _tables(ids, E, pad, rows)):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    if pad == 32 and k <= E:                                   # the layout the grouped GEMMs are tested with
        off, row_token, counts = wl.group_layout(ids, E)
        np.testing.assert_array_equal(t.offsets.cpu().numpy(), off)
        np.testing.assert_array_equal(t.row_token.cpu().numpy()[:off[-1]], row_token)


@pytest.mark.parametrize("T", [40, 3000])
def test_route_tables_without_experts_and_extra_rows(mx, T):
    rng = np.random.default_rng(1)
    ids = rng.integers(-3, 12, (T, 4)).astype(np.int32)        # 8 experts: many ids are none
    ids[0] = [1 << 30, -(1 << 31), 8, -1]
    rows = mx.route_rows(T * 4, 8, 32) + 77
    t = mx.route_tables(torch.from_numpy(ids).cuda(), 8, rows=rows)
    for got, want in zip((t.offsets, t.counts, t.row_token, t.pair_row), _tables(ids, 8, 32, rows)):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    none = mx.route_tables(torch.full((T, 4), -1, dtype=torch.int32, device="cuda"), 8)
    assert none.offsets.abs().sum() == 0 and torch.all(none.row_token == -1) and torch.all(none.pair_row == -1)
    empty = mx.route_tables(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 8)
    assert empty.offsets.tolist() == [0] * 9 and empty.pair_row.shape == (0, 4)
