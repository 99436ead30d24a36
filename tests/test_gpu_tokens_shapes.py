"""The token-level calls at the sizes where their kernels change shape: lanes a
row, pieces in flight, threads a block, chunks with and without a counting
pass."""
import numpy as np
import pytest
import torch

from test_gpu_combine import test_combine_and_gradients as check_combine
from test_gpu_logprobs import _check as check_logprobs, _inputs, test_logprobs_backward as check_logits_gradient
from test_gpu_route import test_route_backward as check_route_gradient, test_route_tables as check_tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H", [64, 65, 128, 129, 256, 257, 511, 512, 513, 1024, 1025, 2048, 2049, 3001])
def test_combine_row_lengths(mx, H, dtype):
    print("combine", H, dtype, flush=True)
    check_combine(mx, 21, 3, 10, H, dtype, True)


@pytest.mark.parametrize("T,k,E", [(1024, 1, 1024), (1025, 1, 4), (1000, 8, 1024), (1024, 8, 513), (8193, 1, 1000),
                                   (2731, 3, 700), (512, 2, 2)])
def test_table_chunks(mx, T, k, E):
    print("tables", T, k, E, flush=True)
    check_tables(mx, T, k, E, 32)


def test_tables_of_one_expert(mx):
    """Every pair to one expert, in the first, in the last and in a middle place."""
    for T in (900, 7000, 40000):
        for e in (0, 77, 127):
            ids = torch.full((T, 1), e, dtype=torch.int32, device="cuda")
            t = mx.route_tables(ids, 128)
            want = np.zeros(128, np.int32)
            want[e] = T
            assert t.counts.cpu().tolist() == want.tolist()
            assert t.pair_row.view(-1).tolist() == list(range(T))
            assert t.row_token[:T].tolist() == list(range(T)) and torch.all(t.row_token[T:] == -1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V,n", [(1024, 2048, 3), (1030, 2056, 0), (1025, 8192, 5), (1024, 8200, 0), (1023, 2048, 5),
                                   (257, 32768, 4), (256, 32776, 4), (256, 65536, 0), (258, 65544, 0), (255, 9000, 2)])
def test_logprobs_block_sizes(mx, T, V, n, dtype):
    print("logprobs", T, V, n, dtype, flush=True)
    x, t = _inputs(T, V, dtype, T + V)
    check_logprobs(mx, x, t, 0.9, n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1023, 1024, 1025, 2047, 2048, 2049, 4096, 4097, 8192, 9000, 16385])
def test_logits_gradient_row_lengths(mx, V, dtype):
    print("gradient", V, dtype, flush=True)
    check_logits_gradient(mx, 5, V, dtype, 0.8, "gh")


@pytest.mark.parametrize("E,k", [(16, 1), (17, 15), (33, 16), (65, 31), (129, 8), (255, 8), (257, 3), (512, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_gradient_sizes(mx, E, k, score):
    print("route gradient", E, k, score, flush=True)
    check_route_gradient(mx, 67, E, k, torch.bfloat16, score, True)


def test_combine_far_rows(mx):
    """Rows whose elements lie past 2^31."""
    rows, H, T = 600000, 4096, 3
    y = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([[rows - 1, 0], [rows - 2, 524288], [5, rows - 3]], dtype=torch.int32, device="cuda")
    g = torch.Generator("cuda").manual_seed(2)
    y[at.long().view(-1)] = torch.randn((2 * T, H), generator=g, device="cuda").bfloat16()
    w = torch.tensor([[0.5, 0.25], [1.0, -1.0], [2.0, 0.125]], device="cuda")        # products exact
    out = mx.moe_combine(y, at, w)
    want = (y[at.long()].float() * w.unsqueeze(2)).sum(1)
    assert torch.equal(out, want.bfloat16())
    row_token = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
    row_token[at.long().view(-1)] = torch.arange(T, device="cuda").repeat_interleave(2)
    d = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    dy, _ = mx.moe_combine_backward(d, y, at, w, row_token)
    assert torch.equal(dy[at.long()], (w.unsqueeze(2) * d.float().unsqueeze(1)).bfloat16())
    dy[at.long().view(-1)] = 0
    assert not dy.view(torch.int16).any()


def test_route_far_rows(mx):
    """A stride that puts the last tokens' logits past 2^31 elements."""
    base = torch.zeros((1 << 21) + 5, 1040, dtype=torch.bfloat16, device="cuda")
    x = base[:, 3:67]
    g = torch.Generator("cuda").manual_seed(3)
    x[-200:] = torch.randn((200, 64), generator=g, device="cuda").bfloat16()
    ids, w = mx.route(x, 4)
    tail_ids, tail_w = mx.route(x[-200:].contiguous(), 4)
    assert torch.equal(ids[-200:], tail_ids) and torch.equal(w[-200:], tail_w)
    assert torch.equal(ids[:4], torch.arange(4, dtype=torch.int32, device="cuda").expand(4, 4))
    dw = torch.randn(w.shape, generator=g, device="cuda")
    d = mx.route_backward(x, ids, dw)
    assert torch.equal(d[-200:], mx.route_backward(x[-200:].contiguous(), tail_ids, dw[-200:].contiguous()))


@pytest.mark.parametrize("dtype,V", [(torch.float32, 100001), (torch.bfloat16, 200003)])
def test_logprobs_larger_than_the_cache(mx, dtype, V):
    """Logits of more than 256 MB: the rows' results are those of a call on a part of them."""
    print("large logits", dtype, V, flush=True)
    x, t = _inputs(720, V, dtype, V)
    for n in (0, 6):
        a, b = mx.token_logprobs(x, t, top_n=n), mx.token_logprobs(x[:300], t[:300], top_n=n)
        for p, q in ((a.logprobs, b.logprobs), (a.entropy, b.entropy), (a.stats, b.stats)) + (
                ((a.top_logprobs, b.top_logprobs), (a.top_ids, b.top_ids)) if n else ()):
            assert torch.equal(p[:300], q)
    g = torch.randn(720, device="cuda")
    d = mx.token_logprobs_backward(x, t, a.stats, a.entropy, g, g)
    part = mx.token_logprobs_backward(x[:150], t[:150], a.stats[:150], a.entropy[:150], g[:150], g[:150])
    assert torch.equal(d[:150], part)
    assert mx.token_logprobs_backward(x, t, a.stats, a.entropy, g, g, out=x) is x and torch.equal(x, d)


@pytest.mark.parametrize("dtype,H", [(torch.float32, 2048), (torch.float32, 1021), (torch.bfloat16, 4099), (torch.bfloat16, 120)])
def test_combine_larger_than_the_cache(mx, dtype, H):
    print("large rows", dtype, H, flush=True)
    size = 2 if dtype is torch.bfloat16 else 4
    rows = (300 << 20) // (H * size)
    y = torch.randn((rows, H), device="cuda").to(dtype)
    T = 500
    at = torch.randperm(rows, device="cuda")[:2 * T].view(T, 2).int()
    w = torch.tensor([0.5, -2.0], device="cuda").expand(T, 2).contiguous()
    out = mx.moe_combine(y, at, w)
    d = torch.randn((T, H), device="cuda").to(dtype)
    row_token = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
    row_token[at.long().view(-1)] = torch.arange(T, device="cuda").repeat_interleave(2)
    dy, dw = mx.moe_combine_backward(d, y, at, w, row_token)
    # the same rows in a small matrix
    small = torch.arange(2 * T, device="cuda").view(T, 2).int()
    ys = y[at.long().view(-1)].contiguous()
    assert torch.equal(out, mx.moe_combine(ys, small, w))
    dys, dws = mx.moe_combine_backward(d, ys, small, w, torch.arange(T, device="cuda").repeat_interleave(2))
    assert torch.equal(dw, dws) and torch.equal(dy[at.long().view(-1)], dys)
    dy[at.long().view(-1)] = 0
    assert not dy.any()
