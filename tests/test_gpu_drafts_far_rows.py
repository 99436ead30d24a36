"""Verification of drafted tokens over rows so far apart that their offsets pass
2^31 elements, in the target's logits, the draft's and the noise."""
import pytest
import torch

from test_gpu_drafts import _case, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_2_31_elements_apart(mx, dtype):
    x, offsets, ids, u, noise, z = _case([1, 2, 0], 4099, dtype, 12)
    ld = (1 << 30) + 3

    def far(t):
        room = torch.zeros((t.shape[0] - 1) * ld + t.shape[1], dtype=t.dtype, device="cuda")
        view = room.as_strided(t.shape, (ld, 1))
        view.copy_(t)
        return view
    assert min(t.shape[0] for t in (x, z, noise)) > 2       # the last row begins past 2^31 elements
    r = _check(mx, far(x), offsets, ids, u, noise, z)
    far_z = far(z)
    far_noise = far(noise)
    again = _check(mx, x, offsets, ids, u, far_noise, far_z)
    assert torch.equal(r.tokens, again.tokens) and torch.equal(r.logprobs, again.logprobs)
