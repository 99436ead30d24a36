"""Outputs over inputs: refused where blocks would read what others write,
right where a call allows it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _tables(mx, T, k, E):
    g = torch.Generator("cuda").manual_seed(T)
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).int()
    return mx.route_tables(ids, E), g


def test_combine_refuses_its_own_rows(mx):
    t, g = _tables(mx, 20, 4, 16)
    y = torch.randn((t.row_token.numel(), 96), generator=g, device="cuda").bfloat16()
    w = torch.rand((20, 4), generator=g, device="cuda")
    keep = y.clone()
    for out in (y[:20], y[7:27], y[-20:]):
        with pytest.raises(mx.MXFP8Error, match="OVERLAP"):
            mx.moe_combine(y, t.pair_row, w, out=out)
    assert torch.equal(y, keep)
    store = torch.empty((y.shape[0] + 20, 96), dtype=y.dtype, device="cuda")       # beside them is fine
    store[20:] = y
    assert torch.equal(mx.moe_combine(store[20:], t.pair_row, w, out=store[:20]), mx.moe_combine(y, t.pair_row, w))


@pytest.mark.parametrize("dtype,H", [(torch.bfloat16, 2048), (torch.bfloat16, 77), (torch.float32, 1001)])
def test_combine_gradients_in_place(mx, dtype, H):
    t, g = _tables(mx, 50, 4, 16)
    y = torch.randn((t.row_token.numel(), H), generator=g, device="cuda").to(dtype)
    w = torch.rand((50, 4), generator=g, device="cuda")
    d = torch.randn((50, H), generator=g, device="cuda").to(dtype)
    dy, dw = mx.moe_combine_backward(d, y, t.pair_row, w, t.row_token)
    from mxfp8_block_scaled_05_amd._tokens import need_rows, stream_of, tokens_lib
    st = tokens_lib().mxfp8_moe_combine_backward(d.data_ptr(), y.data_ptr(), need_rows(y, "y")[0], y.shape[0], H,
                                                 t.pair_row.data_ptr(), w.data_ptr(), t.row_token.data_ptr(), 50, 4,
                                                 y.data_ptr(), w.data_ptr(), stream_of(0))
    assert st == 0 and torch.equal(y, dy) and torch.equal(w, dw)


def test_logits_gradient_refuses_shifted_logits(mx):
    g = torch.Generator("cuda").manual_seed(1)
    store = torch.randn((12, 400), generator=g, device="cuda")
    t = torch.randint(0, 150, (10,), generator=g, device="cuda")
    x = store[:10, :150]
    r = mx.token_logprobs(x, t)
    one = torch.ones(10, device="cuda")
    for out in (store[1:11, :150], store[:10, 1:151], store[2:12, 100:250]):
        with pytest.raises(mx.MXFP8Error, match="OVERLAP"):
            mx.token_logprobs_backward(x, t, r.stats, r.entropy, one, one, out=out)
    d = mx.token_logprobs_backward(x, t, r.stats, r.entropy, one, one)
    beside = store[:10, 150:300]                                                  # between the logits' rows
    assert torch.equal(mx.token_logprobs_backward(x, t, r.stats, r.entropy, one, one, out=beside), d)
    assert torch.equal(mx.token_logprobs_backward(x, t, r.stats, r.entropy, one, one, out=x), d)
