"""Verification of drafted tokens over rows longer than any vocabulary.

Where a row rises slowly every group of columns brings a new maximum, and the
sum so far is scaled by an exponential each time.  Its error is one rounding,
2^-24 and less, but of one sign: over 4096 such steps they come to 2^-14, more than
the bounds with which the decisions are taken.  So a row is cut into slices of
at most 2^18 columns, 70 steps, and those are joined in fp64: the sum is within
2^-16.2 of its value (drafts.hip), and log p within that and half a step of fp32."""
import pytest
import torch

from test_gpu_drafts import _case, _check

pytestmark = pytest.mark.gpu


def test_rows_that_rise_slowly(mx):
    V, B, n = 1 << 24, 8, 31
    R = B * (n + 1)                                         # as many rows as compute units: none is cut for their sake
    step = 0.9 * 2.0 ** -25                                 # e^-step is 1 in fp32
    row = (torch.arange(V, device="cuda") // 4096).double().mul_(step).float()
    x = row.expand(R, V).contiguous()
    z = row.double()
    z -= z.max()
    logp = z - torch.log(torch.exp(z).sum())
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    ids = torch.randint(0, V, (B * n,), generator=g, device="cuda")
    # every second request stops at its 20th draft, by 2^-17 of p; the others take all of theirs, by as much
    p = torch.exp(logp[ids])
    u = (p * (1 - 2.0 ** -17)).float()
    stop = torch.arange(0, B, 2, device="cuda") * n + 19
    u[stop] = (p[stop] * (1 + 2.0 ** -17)).float()
    noise = torch.empty((B, V), device="cuda").exponential_(generator=g).clamp_min_(2.0 ** -30)
    offsets = torch.arange(0, R + 1, n + 1, dtype=torch.int32, device="cuda")
    r = mx.verify_drafts(x, offsets, ids, u, noise)
    assert r.accepted.tolist() == [19 if b % 2 == 0 else n for b in range(B)]
    for b in range(B):
        end, lo = int(r.accepted[b]), b * (n + 1)
        score = torch.exp(logp) / noise[b].double()
        if end < n:
            score[ids[b * n + end]] = 0
        tokens = ids[b * n:b * n + end].tolist() + [int(torch.nonzero(score == score.max())[0])]
        assert r.tokens[lo:lo + n + 1].tolist() == tokens + [-1] * (n - end)
        want = logp[torch.tensor(tokens, device="cuda")]
        got = r.logprobs[lo:lo + end + 1].double()
        assert bool(((got - want).abs() <= 2.0 ** -16.2 + 2.0 ** -24 * want.abs()).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_more_slices_than_a_wave_has_lanes(mx, dtype):
    """Slices at their longest, joined in rounds, by few rows and by many"""
    _check(mx, *_case([1], 17_000_003, dtype, 3))
    _check(mx, *_case([1] * 88, 300_007, dtype, 4))         # 264 rows, two slices each
