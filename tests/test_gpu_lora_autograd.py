"""The adapters' calls write y and d_x in place: autograd hears of it, as of
torch's own in-place operations."""
import pytest
import torch

from test_gpu_lora import _gen, _ids, _whole

pytestmark = pytest.mark.gpu

T, E, r, K, N = 40, 2, 8, 64, 64


def _inputs(mx):
    g = _gen(1)
    tables = mx.route_tables(_ids(T, E, 1).view(-1, 1), E)
    return _whole((T, K), g, 1), _whole((E, r, K), g, 1), _whole((E, N, r), g, 1), tables


def test_values_that_autograd_needs_are_not_replaced_unseen(mx):
    x, a, b, tables = _inputs(mx)
    w = torch.ones((T, N), device="cuda", requires_grad=True)
    y = w * 2
    loss = (y * y).sum()                                    # needs y as it is now
    mx.lora_add_(y.detach(), x, a, b, tables)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    d = torch.ones((T, K), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    d_x = d * 2
    loss = (d_x * d_x).sum()
    hidden = torch.zeros((tables.row_token.numel(), r), device="cuda")
    mx.lora_backward_(d_x.detach(), b[0, :, :1].t().expand(T, N).contiguous(), x, a, b, hidden, tables)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_versions_count_what_is_written(mx):
    x, a, b, tables = _inputs(mx)
    y = torch.zeros((T, N), device="cuda")
    d_x = torch.zeros((T, K), device="cuda", dtype=torch.bfloat16)
    hidden = mx.lora_add_(y, x, a, b, tables, keep_hidden=True)
    before = [t._version for t in (x, a, b, hidden)]
    mx.lora_backward_(d_x, y.to(torch.bfloat16), x, a, b, hidden, tables)
    mx.lora_backward_(None, y.to(torch.bfloat16), x, a, b, hidden, tables)
    assert (y._version, d_x._version) == (1, 1)
    assert [t._version for t in (x, a, b, hidden)] == before
    with torch.inference_mode():
        y = torch.zeros((T, N), device="cuda")
        mx.lora_add_(y, x, a, b, tables)
    with pytest.raises(ValueError):
        mx.lora_add_(d_x[:, :32], x, a, b, tables)
    assert d_x._version == 1                                # a refused call has written nothing
