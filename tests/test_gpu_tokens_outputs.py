"""Every element of every output is written: the calls get outputs full of NaN
or of all bits set, in place of what an allocator happens to hand out."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

CODE = {torch.float32: 0, torch.bfloat16: 1}


def _lib():
    from mxfp8_block_scaled_05_amd._tokens import stream_of, tokens_lib
    return tokens_lib(), stream_of(0)


def _filled(shape, dtype):
    """All bits set: a NaN, or -1 as an integer; 256 more elements behind it show a write past the end."""
    n = int(np.prod(shape))
    raw = torch.full(((n + 256) * torch.empty((), dtype=dtype).element_size(),), 255, dtype=torch.uint8, device="cuda")
    all_of = raw.view(dtype)
    return all_of[:n].view(shape), raw[n * all_of.element_size():]


def _untouched(*tails):
    return all(bool((t == 255).all()) for t in tails)


def _combine_backward(mx, d, y, pair_row, w, row_token):
    L, stream = _lib()
    dy, tail = _filled(y.shape, y.dtype)
    dw, tail2 = _filled(w.shape, torch.float32)
    st = L.mxfp8_moe_combine_backward(d.data_ptr(), y.data_ptr(), CODE[y.dtype], y.shape[0], y.shape[1], pair_row.data_ptr(),
                                      w.data_ptr(), row_token.data_ptr(), *w.shape, dy.data_ptr(), dw.data_ptr(), stream)
    assert st == 0 and _untouched(tail, tail2)
    return dy, dw


def _combine(mx, y, pair_row, w):
    L, stream = _lib()
    out, tail = _filled((w.shape[0], y.shape[1]), y.dtype)
    st = L.mxfp8_moe_combine(y.data_ptr(), CODE[y.dtype], *y.shape, pair_row.data_ptr(), w.data_ptr(), *w.shape,
                             out.data_ptr(), stream)
    assert st == 0 and _untouched(tail)
    return out


@pytest.mark.parametrize("T,k,E,H", [(1, 8, 128, 2048), (33, 10, 64, 1001), (257, 2, 9, 77), (100, 17, 40, 264), (7, 4, 8, 7),
                                     (2000, 8, 128, 136)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_combine(mx, T, k, E, H, dtype):
    print("combine", T, k, E, H, dtype, flush=True)
    g = torch.Generator("cuda").manual_seed(H)
    ids = torch.randint(-2, E, (T, k), generator=g, device="cuda").int()
    t = mx.route_tables(ids, E)
    y = torch.randn((t.row_token.numel(), H), generator=g, device="cuda").to(dtype)
    w = torch.rand((T, k), generator=g, device="cuda")
    d = torch.randn((T, H), generator=g, device="cuda").to(dtype)
    dy, dw = _combine_backward(mx, d, y, t.pair_row, w, t.row_token)
    assert bool((dy[t.row_token < 0] == 0).all()) and bool((dw[t.pair_row < 0] == 0).all())
    token = t.row_token.clamp_min(0)
    real = t.row_token >= 0
    weight = torch.zeros(y.shape[0], device="cuda")
    weight[t.pair_row[t.pair_row >= 0].long()] = w[t.pair_row >= 0]
    want = (weight.unsqueeze(1) * d[token].float()).to(dtype)              # one fp32 product, one rounding
    assert torch.equal(dy[real], want[real]) and torch.isfinite(dw).all()
    out = _combine(mx, y, t.pair_row, w)
    assert torch.equal(out, mx.moe_combine(y, t.pair_row, w)) and torch.isfinite(out).all()


@pytest.mark.parametrize("dtype,rows,H", [(torch.bfloat16, 600000, 4096), (torch.float32, 40000, 2048), (torch.bfloat16, 39000, 4099)])
def test_combine_zeros_far_and_many_rows(mx, dtype, rows, H):
    """Past 2^31 elements, and more than the last-level cache holds: all rows but 6 are padding."""
    print("far rows", rows, H, dtype, flush=True)
    T = 3
    g = torch.Generator("cuda").manual_seed(2)
    at = torch.tensor([[rows - 1, 0], [rows - 2, rows // 2], [5, rows - 3]], dtype=torch.int32, device="cuda")
    y = torch.full((rows, H), float("nan"), dtype=dtype, device="cuda")     # padding rows are never read
    y[at.long().view(-1)] = torch.randn((2 * T, H), generator=g, device="cuda").to(dtype)
    w = torch.tensor([[0.5, 0.25], [1.0, -1.0], [2.0, 0.125]], device="cuda")
    row_token = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
    row_token[at.long().view(-1)] = torch.arange(T, device="cuda").repeat_interleave(2)
    d = torch.randn((T, H), generator=g, device="cuda").to(dtype)
    dy, dw = _combine_backward(mx, d, y, at, w, row_token)
    assert torch.equal(dy[at.long()], (w.unsqueeze(2) * d.float().unsqueeze(1)).to(dtype)) and torch.isfinite(dw).all()
    dy[at.long().view(-1)] = 0
    for part in dy.split(1 << 16):
        assert not part.view(torch.uint8).any()


@pytest.mark.parametrize("T,k,E,pad", [(1, 1, 1, 32), (32, 8, 128, 32), (7, 3, 1024, 1), (171, 3, 5, 128), (1500, 7, 61, 32),
                                       (16384, 8, 256, 32), (70001, 1, 2, 1), (9000, 10, 1024, 128)])
def test_tables(mx, T, k, E, pad):
    print("tables", T, k, E, pad, flush=True)
    L, stream = _lib()
    g = torch.Generator("cuda").manual_seed(T)
    ids = torch.randint(-1, E, (T, k), generator=g, device="cuda").int()
    rows = mx.route_rows(T * k, E, pad) + 33
    off, t1 = _filled((E + 1,), torch.int32)
    cnt, t2 = _filled((E,), torch.int32)
    tok, t3 = _filled((rows,), torch.int64)
    tok.fill_(1 << 40)
    pr, t4 = _filled((T, k), torch.int32)
    pr.fill_(1 << 30)
    need = L.mxfp8_route_tables_workspace_bytes(T, k, E)
    ws, t5 = _filled((max(need // 4, 1),), torch.int32)
    st = L.mxfp8_route_tables(ids.data_ptr(), T, k, E, pad, off.data_ptr(), cnt.data_ptr(), tok.data_ptr(), rows, pr.data_ptr(),
                              ws.data_ptr() if need else None, need, stream)
    assert st == 0 and _untouched(t1, t2, t3, t4, t5)
    flat = ids.view(-1).cpu().numpy()
    counts = np.bincount(flat[flat >= 0], minlength=E)
    offsets = np.concatenate(([0], np.cumsum((counts + pad - 1) // pad * pad)))
    np.testing.assert_array_equal(off.cpu().numpy(), offsets)
    np.testing.assert_array_equal(cnt.cpu().numpy(), counts)
    order = np.argsort(flat, kind="stable")
    order = order[flat[order] >= 0]
    first = np.concatenate(([0], np.cumsum(counts)))[:-1]
    row = offsets[flat[order]] + np.arange(order.size) - first[flat[order]]
    want_tok, want_pr = np.full(rows, -1, np.int64), np.full(T * k, -1, np.int64)
    want_tok[row] = order // k
    want_pr[order] = row
    np.testing.assert_array_equal(tok.cpu().numpy(), want_tok)
    np.testing.assert_array_equal(pr.view(-1).cpu().numpy(), want_pr)


@pytest.mark.parametrize("T,V,n", [(1, 131072, 20), (3, 50, 5), (300, 9001, 0), (1100, 700, 4), (260, 70001, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logprobs(mx, T, V, n, dtype):
    print("logprobs", T, V, n, dtype, flush=True)
    L, stream = _lib()
    g = torch.Generator("cuda").manual_seed(V)
    x = (torch.randn((T, V), generator=g, device="cuda") * 2).to(dtype)
    t = torch.randint(-1, V, (T,), generator=g, device="cuda")
    want = mx.token_logprobs(x, t, top_n=n)
    lp, t1 = _filled((T,), torch.float32)
    H, t2 = _filled((T,), torch.float32)
    st, t3 = _filled((T, 2), torch.float32)
    tl, t4 = _filled((T, n), torch.float32)
    ti, t5 = _filled((T, n), torch.int64)
    need = L.mxfp8_token_logprobs_workspace_bytes(T, V, n)
    ws, t6 = _filled((max(need // 4, 1),), torch.float32)
    assert L.mxfp8_token_logprobs(x.data_ptr(), CODE[dtype], V, T, V, t.data_ptr(), 1.0, n, lp.data_ptr(), H.data_ptr(),
                                  st.data_ptr(), tl.data_ptr() if n else None, ti.data_ptr() if n else None,
                                  ws.data_ptr() if need else None, need, stream) == 0
    assert _untouched(t1, t2, t3, t4, t5, t6)
    assert torch.equal(lp, want.logprobs) and torch.equal(H, want.entropy) and torch.equal(st, want.stats)
    if n:
        assert torch.equal(tl, want.top_logprobs) and torch.equal(ti, want.top_ids)
    d, tail = _filled((T, V), dtype)
    one = torch.ones(T, device="cuda")
    assert L.mxfp8_token_logprobs_backward(x.data_ptr(), CODE[dtype], V, T, V, t.data_ptr(), st.data_ptr(), H.data_ptr(),
                                           one.data_ptr(), one.data_ptr(), 1.0, d.data_ptr(), V, stream) == 0
    assert _untouched(tail) and torch.isfinite(d).all()
    assert torch.equal(d, mx.token_logprobs_backward(x, t, want.stats, want.entropy, one, one))


@pytest.mark.parametrize("T,E,k", [(1, 8, 1), (65, 128, 8), (33, 511, 31), (100, 37, 5)])
@pytest.mark.parametrize("score", [0, 1])
def test_route(mx, T, E, k, score):
    print("route", T, E, k, score, flush=True)
    L, stream = _lib()
    g = torch.Generator("cuda").manual_seed(E)
    x = torch.randn((T, E), generator=g, device="cuda")
    ids, t1 = _filled((T, k), torch.int32)
    w, t2 = _filled((T, k), torch.float32)
    d, t3 = _filled((T, E), torch.float32)
    assert L.mxfp8_route(x.data_ptr(), 0, E, T, E, k, score, None, 1, 1, 1, 1, 1.0, ids.data_ptr(), w.data_ptr(), stream) == 0
    assert L.mxfp8_route_backward(x.data_ptr(), 0, E, T, E, k, score, ids.data_ptr(), w.data_ptr(), 1, 1.0, d.data_ptr(), stream) == 0
    assert _untouched(t1, t2, t3)
    assert int(ids.min()) >= 0 and int(ids.max()) < E and torch.isfinite(w).all() and torch.isfinite(d).all()
