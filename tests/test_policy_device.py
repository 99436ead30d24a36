"""The calls of include/mxfp8_policy.h launch on the current device: tensors of
another one are refused, not handed to it by their addresses."""
import pytest

from mxfp8_block_scaled_05_amd import _policy, checkpoint, drafts, lora


def test_streams_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(_policy, "_current_device", lambda: 2)
    monkeypatch.setattr(_policy, "_stream_of", lambda device: 1000 + device)
    assert _policy.stream_of(2) == 1002
    for other in (0, 1, 3):
        with pytest.raises(ValueError, match="cuda:%d.*cuda:2" % other):
            _policy.stream_of(other)
    assert checkpoint.stream_of is lora.stream_of is drafts.stream_of is _policy.stream_of


@pytest.mark.gpu
def test_calls_refuse_tensors_of_another_device(mx, monkeypatch):
    """The tensors' device is 0 and the current one said to be 1: every call raises before it writes."""
    import torch
    T, E, r, K, N = 32, 1, 8, 64, 64
    gu = torch.randn((T, 2 * K), device="cuda").to(torch.bfloat16)
    saved = mx.swiglu(gu)
    tables = mx.route_tables(torch.zeros((T, 1), dtype=torch.int32, device="cuda"), E)
    x, d_x, y = (torch.ones((T, n), dtype=torch.bfloat16, device="cuda") for n in (K, K, N))
    a, b = (torch.ones(s, dtype=torch.bfloat16, device="cuda") for s in ((E, r, K), (E, N, r)))
    hidden = torch.ones((tables.row_token.numel(), r), device="cuda")
    logits, noise = torch.zeros((2, 16), device="cuda"), torch.ones((1, 16), device="cuda")
    offsets = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    ids, u = torch.zeros(1, dtype=torch.long, device="cuda"), torch.zeros(1, device="cuda")
    calls = (lambda: mx.swiglu(gu), lambda: mx.swiglu_backward(x, saved.saved_q, saved.saved_s), lambda: mx.lora_add_(y, x, a, b, tables),
             lambda: mx.lora_backward_(d_x, y, x, a, b, hidden, tables), lambda: mx.verify_drafts(logits, offsets, ids, u, noise))
    monkeypatch.setattr(_policy, "_current_device", lambda: 1)
    for call in calls:
        with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
            call()
    monkeypatch.undo()
    assert bool((y == 1).all()) and bool((d_x == 1).all())
    for call in calls:
        call()
    assert bool((y != 1).all()) and bool((d_x != 1).all())
