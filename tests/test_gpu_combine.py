"""Expert rows back in token order, and the gradients, against fp64."""
import numpy as np
import pytest
import torch

import workloads as wl

pytestmark = pytest.mark.gpu

HALF32 = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def _setup(mx, T, k, E, H, dtype, drop=False):
    rng = np.random.default_rng(T + H)
    ids = wl.zipf_topk_routing(rng, T, E, k)
    if drop:
        ids[::3, 0] = -1
        ids[0] = -1                                            # a token with no expert at all
    t = mx.route_tables(torch.from_numpy(ids).cuda(), E)
    g = torch.Generator("cuda").manual_seed(H)
    y = torch.randn((t.row_token.numel(), H), generator=g, device="cuda").to(dtype)
    w = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), 1)
    d = torch.randn((T, H), generator=g, device="cuda").to(dtype)
    return t, y, w, d


CASES = [(1, 1, 8, 1, torch.float32, False), (1, 8, 128, 2048, torch.bfloat16, False),
         (16, 8, 128, 2048, torch.bfloat16, False), (33, 10, 64, 1001, torch.bfloat16, True),
         (257, 2, 9, 77, torch.float32, True), (100, 17, 40, 264, torch.bfloat16, False),
         (50, 3, 8, 4096, torch.float32, False), (7, 4, 8, 7, torch.bfloat16, True), (5, 2, 4, 20001, torch.bfloat16, False)]


@pytest.mark.parametrize("T,k,E,H,dtype,drop", CASES)
def test_combine_and_gradients(mx, T, k, E, H, dtype, drop):
    t, y, w, d = _setup(mx, T, k, E, H, dtype, drop)
    pr = t.pair_row.long().cpu()
    yd, wd, dd = y.double().cpu(), w.double().cpu(), d.double().cpu()
    real = (pr >= 0).double()
    rows = yd[pr.clamp_min(0)] * real.unsqueeze(2)              # [T, k, H]

    out = mx.moe_combine(y, t.pair_row, w)
    want = (rows * wd.unsqueeze(2)).sum(1)
    size = (rows * wd.unsqueeze(2)).abs().sum(1)
    err = (out.double().cpu() - want).abs()
    assert out.dtype == dtype and bool((err <= k * HALF32 * size + HALF[dtype] * want.abs() * (1 + 1e-3)).all())

    dy, dw = mx.moe_combine_backward(d, y, t.pair_row, w, t.row_token)
    want_dw = (rows * dd.unsqueeze(1)).sum(2)
    size = (rows * dd.unsqueeze(1)).abs().sum(2)
    # a lane adds every 64th 16-byte piece, then six steps over the lanes
    adds = H / 64 + 8 + 6
    assert bool(((dw.double().cpu() - want_dw).abs() <= adds * HALF32 * size).all())
    want_dy = torch.zeros_like(yd)
    flat = pr.view(-1)
    keep = flat >= 0
    want_dy[flat[keep]] = (wd.unsqueeze(2) * dd.unsqueeze(1)).view(-1, H)[keep]
    # the fp32 product, then one rounding
    assert bool(((dy.double().cpu() - want_dy).abs() <= (HALF[dtype] + 2 * HALF32) * want_dy.abs()).all())
    # padding rows: exactly zero, whatever the memory held
    assert bool((dy.cpu()[t.row_token.cpu() < 0] == 0).all())


def test_combine_leaves_padding_rows_alone_and_takes_views(mx):
    t, y, w, d = _setup(mx, 20, 4, 16, 96, torch.bfloat16)
    out = mx.moe_combine(y, t.pair_row, w)
    dy, dw = mx.moe_combine_backward(d, y, t.pair_row, w, t.row_token)
    y[t.row_token < 0] = float("nan")                          # unwritten rows of a grouped GEMM's output
    assert torch.equal(mx.moe_combine(y, t.pair_row, w), out)
    dy2, dw2 = mx.moe_combine_backward(d, y, t.pair_row, w, t.row_token)
    assert torch.equal(dy, dy2) and torch.equal(dw, dw2)
    # a view that starts off a 16-byte boundary
    flat = torch.empty(y.numel() + 3, dtype=y.dtype, device="cuda")
    v = flat[3:].view_as(y)
    v.copy_(y)
    assert torch.equal(mx.moe_combine(v, t.pair_row, w), out)
    # rows outside y: nothing is added, no gradient
    pr = t.pair_row.clone()
    pr[3] = torch.tensor([-1, y.shape[0], 1 << 30, -(1 << 31)], dtype=torch.int32, device="cuda")
    assert torch.all(mx.moe_combine(y, pr, w)[3] == 0)
    assert torch.all(mx.moe_combine_backward(d, y, pr, w, t.row_token)[1][3] == 0)
    none = mx.moe_combine(y, pr[:0], w[:0])
    assert none.shape == (0, 96)


def test_combine_checks(mx):
    t, y, w, d = _setup(mx, 4, 2, 8, 64, torch.bfloat16)
    for bad in (lambda: mx.moe_combine(y, t.pair_row, w[:2]), lambda: mx.moe_combine(y[0], t.pair_row, w),
                lambda: mx.moe_combine(y[:, ::2], t.pair_row, w), lambda: mx.moe_combine(y, t.pair_row, w, out=y),
                lambda: mx.moe_combine_backward(d[:1], y, t.pair_row, w, t.row_token),
                lambda: mx.moe_combine_backward(d, y, t.pair_row, w, t.row_token[:3])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        mx.moe_combine(y.half(), t.pair_row, w)
    with pytest.raises(TypeError):
        mx.moe_combine(y, t.pair_row.long(), w)
    with pytest.raises(mx.MXFP8Error):
        mx.route(torch.zeros((2, 8), device="cuda"), 9)
    with pytest.raises(ValueError):
        mx.route(torch.zeros((2, 8), device="cuda"), 2, score="linear")
