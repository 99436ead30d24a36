"""Rows 2^31 and more elements apart, as the last positions of [batch, length,
vocabulary] logits are."""
import pytest
import torch

pytestmark = pytest.mark.gpu

FAR = (1 << 31) + 24


def _far(rows, cols):
    store = torch.empty(FAR * (rows - 1) + cols, dtype=torch.bfloat16, device="cuda")
    return torch.as_strided(store, (rows, cols), (FAR, 1))


def test_logprobs_of_far_rows(mx):
    g = torch.Generator("cuda").manual_seed(1)
    src = (torch.randn((3, 20001), generator=g, device="cuda") * 2).bfloat16()
    x = _far(3, 20001)
    x.copy_(src)
    t = torch.tensor([5, -100, 20000], device="cuda")
    a, b = mx.token_logprobs(x, t, top_n=4), mx.token_logprobs(src, t, top_n=4)
    for p, q in ((a.logprobs, b.logprobs), (a.entropy, b.entropy), (a.stats, b.stats), (a.top_ids, b.top_ids),
                 (a.top_logprobs, b.top_logprobs)):
        assert torch.equal(p, q)
    one = torch.ones(3, device="cuda")
    d = mx.token_logprobs_backward(src, t, b.stats, b.entropy, one, one)
    assert torch.equal(mx.token_logprobs_backward(x, t, a.stats, a.entropy, one, one), d)
    assert mx.token_logprobs_backward(x, t, a.stats, a.entropy, one, one, out=x) is x and torch.equal(x, d)


def test_route_of_far_rows(mx):
    g = torch.Generator("cuda").manual_seed(2)
    src = torch.randn((3, 61), generator=g, device="cuda").bfloat16()
    x = _far(3, 61)
    x.copy_(src)
    ids, w = mx.route(src, 5)
    ids2, w2 = mx.route(x, 5)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    assert torch.equal(mx.route_backward(x, ids, w), mx.route_backward(src, ids, w))
