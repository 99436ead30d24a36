"""Verification of drafted tokens on the GPU against the rule itself in fp64.

Accepted counts and tokens have to be equal: decisions that fp32 could get
wrong are part of the tests.  Log-probabilities: the row's sum is within 2^-17
of its value (drafts.hip), so log p is within 2^-16 and half a step of fp32.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _softmax(x, temperature):
    """(p, log p) in fp64; NaN where there is no distribution"""
    z = x.double() / temperature
    z = z - z.amax(-1, keepdim=True)
    e = torch.exp(z)
    s = e.sum(-1, keepdim=True)
    return e / s, z - torch.log(s)


def _want(logits, offsets, ids, u, noise, draft_logits, temperature):
    """(accepted, tokens, logprobs) of the rule, request by request"""
    p, logp = _softmax(logits, temperature)
    q = None if draft_logits is None else _softmax(draft_logits, temperature)[0]
    p, logp, noise = p.cpu(), logp.cpu(), noise.double().cpu()
    q = None if q is None else q.cpu()
    ids, u, V = ids.tolist(), u.double().tolist(), logits.shape[1]
    B, R = len(offsets) - 1, logits.shape[0]
    accepted, tokens, lps = [], [-1] * R, [0.0] * R

    def race(w, b):
        ok = (w > 0) & (w / noise[b] > 0)
        if not bool(ok.any()):
            return -1
        score = torch.where(ok, w / noise[b], -1.0)
        return int(torch.nonzero(score == score.max())[0])
    for b in range(B):
        lo, n = offsets[b], offsets[b + 1] - offsets[b] - 1
        if n < 0:
            accepted.append(0)
            continue
        end = n
        for i in range(n):
            x, d = ids[lo - b + i], lo - b + i
            px = p[lo + i, x].item() if 0 <= x < V else float("nan")
            qx = 1.0 if q is None else q[d, x].item() if 0 <= x < V else 0.0
            if not u[d] * qx < px:
                end = i
                break
            tokens[lo + i], lps[lo + i] = x, logp[lo + i, x].item()
        row, w = lo + end, p[lo + end]
        token = -1
        if end < n:
            if q is None:
                r = w.clone()
                if 0 <= ids[lo - b + end] < V:
                    r[ids[lo - b + end]] = 0
            else:
                r = w - q[lo - b + end]
            token = race(r, b)
        if token < 0:
            token = race(w, b)
        tokens[row] = token
        lps[row] = logp[row, token].item() if token >= 0 else float("nan")
        accepted.append(end)
    return torch.tensor(accepted, dtype=torch.int32), torch.tensor(tokens), torch.tensor(lps, dtype=torch.float64)


def _check(mx, logits, offsets, ids, u, noise, draft=None, temperature=1.0):
    r = mx.verify_drafts(logits, torch.tensor(offsets, dtype=torch.int32, device="cuda"), ids, u, noise, draft_logits=draft,
                         temperature=temperature)
    accepted, tokens, lps = _want(logits, offsets, ids, u, noise, draft, temperature)
    assert r.accepted.cpu().tolist() == accepted.tolist()
    assert r.tokens.cpu().tolist() == tokens.tolist()
    got = r.logprobs.double().cpu()
    assert torch.equal(got.isnan(), lps.isnan())
    real = ~lps.isnan()
    assert bool(((got - lps).abs()[real] <= 2.0 ** -16 + 2.0 ** -24 * lps.abs()[real]).all())
    return r


def _case(counts, V, dtype, seed, draft=True, temperature=1.0, noise_of_draft=0.7):
    g = _gen(seed)
    B, D = len(counts), sum(counts)
    offsets = [0]
    for n in counts:
        offsets.append(offsets[-1] + n + 1)
    R = B + D
    x = torch.randn((R, V), generator=g, device="cuda") * 2.5
    last = torch.tensor(offsets[1:], device="cuda") - 1
    drafted = torch.ones(R, dtype=torch.bool, device="cuda")
    drafted[last] = False
    z = (x[drafted] + torch.randn((D, V), generator=g, device="cuda") * noise_of_draft).to(dtype)
    race = torch.empty((D, V), device="cuda").exponential_(generator=g)
    ids = torch.argmax(z.float() / temperature - torch.log(race), 1) if D else torch.zeros(0, dtype=torch.long, device="cuda")
    u = torch.rand(D, generator=g, device="cuda")
    noise = torch.empty((B, V), device="cuda").exponential_(generator=g).clamp_min_(2.0 ** -24)
    return x.to(dtype), offsets, ids, u, noise, (z if draft else None)


COUNTS = [[0], [4], [1, 0, 7, 3], [2] * 40, [0] * 9, [13, 0, 1]]
SIZES = [1, 2, 7, 64, 257, 4095, 4104, 20001]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("which", range(len(COUNTS)))
def test_against_the_rule(mx, which, V, dtype):
    for draft in (True, False):
        for t in (1.0, 0.6):
            _check(mx, *_case(COUNTS[which], V, dtype, 100 * which + V % 97, draft, t), temperature=t)


@pytest.mark.parametrize("counts,V", [([40, 2, 31, 32], 300), ([100], 5000), ([4], 131072), ([3, 0, 5, 1], 100003), ([2] * 300, 1000), ([1] * 700, 999), ([5] * 30, 70001)])
def test_larger(mx, counts, V):
    for dtype in (torch.float32, torch.bfloat16):
        _check(mx, *_case(counts, V, dtype, V % 1000))


def test_one_row_larger_than_the_last_level_cache(mx):
    """70 million columns: slices of a row past what one block takes, offsets in bytes past 2^31 over the rows"""
    V = 70_000_001
    case = _case([6], V, torch.bfloat16, 5)
    assert case[0].numel() * 2 + case[5].numel() * 2 > 1 << 30
    _check(mx, *case)


def test_decisions_that_fp32_cannot_take(mx):
    """Uniforms at p / q itself and one step of fp32 to both sides: the order is that of fp64."""
    V = 50
    x, offsets, ids, u, noise, z = _case([1] * 600, V, torch.float32, 3)
    drafted = torch.arange(0, 1200, 2, device="cuda")
    p = _softmax(x, 1.0)[0][drafted, ids]
    q = _softmax(z, 1.0)[0].gather(1, ids.unsqueeze(1)).squeeze(1)
    close = (p / q).float()
    below = close < 1
    step = torch.tensor([-1, 0, 1], device="cuda").repeat(200)
    moved = (close.view(torch.int32) + step.to(torch.int32)).view(torch.float32)
    u = torch.where(below, moved, u)
    assert int(below.sum()) > 150
    r = _check(mx, x, offsets, ids, u, noise, z)
    assert 0 < int(r.accepted.sum()) < 600


def test_races_that_fp32_cannot_take(mx):
    """Two columns with equal scores, and scores a step of fp32 apart"""
    V, B = 300, 400
    g = _gen(8)
    x = torch.randn((B, V), generator=g, device="cuda") - 6
    noise = torch.empty((B, V), device="cuda").exponential_(generator=g).clamp_min_(1e-3)
    first = torch.randint(0, V // 2, (B,), generator=g, device="cuda")
    second = first + torch.randint(1, V // 2, (B,), generator=g, device="cuda")
    row = torch.arange(B, device="cuda")
    x[row, first], x[row, second] = 3.0, 3.0
    value = torch.rand(B, generator=g, device="cuda") * 0.2 + 0.01
    step = torch.tensor([-1, 0, 0, 1], device="cuda", dtype=torch.int32).repeat(B // 4)
    noise[row, first] = value
    noise[row, second] = (value.view(torch.int32) + step).view(torch.float32)
    ids, u = torch.zeros(0, dtype=torch.long, device="cuda"), torch.zeros(0, device="cuda")
    r = _check(mx, x, list(range(B + 1)), ids, u, noise)
    tied = step == 0
    assert torch.equal(r.tokens[tied], first[tied]) and torch.equal(r.tokens[step == -1], second[step == -1])
    # the same with a draft whose probabilities leave tiny differences
    x2 = torch.randn((2 * B, V), generator=g, device="cuda")
    z = x2[::2].clone()
    z[row, first] -= 1e-4
    z[row, second] -= 1e-4
    u = torch.full((B,), 0.9999999, device="cuda")
    worst = torch.argmin(x2[::2], 1)
    _check(mx, x2, list(range(0, 2 * B + 1, 2)), worst, u, noise, z)


def test_same_distributions_accept_everything(mx):
    x, offsets, ids, u, noise, _ = _case([3] * 20, 500, torch.bfloat16, 4)
    drafted = torch.ones(80, dtype=torch.bool, device="cuda")
    drafted[3::4] = False
    u[:] = 1 - 2.0 ** -24
    r = _check(mx, x, offsets, ids, u, noise, x[drafted].contiguous())
    assert bool((r.accepted == 3).all())
    # u = 1 refuses, nothing is left of p - q, and the token comes from p
    u[0] = 1.0
    r = _check(mx, x, offsets, ids, u, noise, x[drafted].contiguous())
    assert r.accepted[0] == 0 and r.tokens[0] >= 0


def test_distribution_of_the_first_token(mx):
    """What comes out first is distributed as the target, whatever the draft: 200000 requests, each column within six
    standard deviations."""
    N, V = 200_000, 6
    g = _gen(1)
    p_logits = torch.tensor([0.3, -1.0, 1.2, 0.0, -2.5, 0.9], device="cuda")
    q_logits = torch.tensor([1.0, 0.4, -0.3, -math.inf, 0.5, 0.2], device="cuda")
    x, z = p_logits.repeat(2 * N, 1), q_logits.repeat(N, 1)
    offsets = torch.arange(0, 2 * N + 1, 2, dtype=torch.int32, device="cuda")
    race = torch.empty((N, V), device="cuda").exponential_(generator=g)
    ids = torch.argmax(z - torch.log(race), 1)
    u = torch.rand(N, generator=g, device="cuda")
    noise = torch.empty((N, V), device="cuda").exponential_(generator=g)
    p = torch.softmax(p_logits.double(), 0)
    for draft, tokens in ((z, ids), (None, torch.full_like(ids, 2))):
        r = mx.verify_drafts(x, offsets, tokens, u, noise, draft_logits=draft)
        share = torch.bincount(r.tokens[::2], minlength=V).double() / N
        assert bool(((share - p).abs() <= 6 * torch.sqrt(p * (1 - p) / N)).all())
        second = torch.bincount(r.tokens[1::2][r.accepted == 1], minlength=V).double()
        n = second.sum()
        assert bool(((second / n - p).abs() <= 6 * torch.sqrt(p * (1 - p) / n)).all())


def test_greedy_by_temperature(mx):
    """A temperature near 0 compares with the largest logit"""
    x, offsets, ids, u, noise, _ = _case([4] * 30, 800, torch.bfloat16, 6)
    best = torch.argmax(x.float(), 1)
    drafted = torch.ones(150, dtype=torch.bool, device="cuda")
    drafted[4::5] = False
    g = _gen(3)
    ids = torch.where(torch.rand(120, generator=g, device="cuda") < 0.7, best[drafted], ids)
    x.scatter_add_(1, best.unsqueeze(1), torch.ones((150, 1), dtype=x.dtype, device="cuda"))       # no equal maxima
    for t in (2.0 ** -60, 1e-3):
        r = mx.verify_drafts(x, torch.tensor(offsets, dtype=torch.int32, device="cuda"), ids, u, noise, temperature=t)
        right = (ids == best[drafted]).view(30, 4).int().cumprod(1).sum(1)
        assert torch.equal(r.accepted.long(), right.long())
        at = torch.tensor(offsets[:-1], device="cuda") + right
        assert torch.equal(r.tokens[at], best[at])


def test_masked_and_unusual_logits(mx):
    """Columns of -Inf and of the type's lowest value; rows of nothing else; NaN and +Inf in a row."""
    inf = float("inf")
    for dtype in (torch.float32, torch.bfloat16):
        x, offsets, ids, u, noise, z = _case([3] * 12, 130, dtype, 7)
        lowest = torch.finfo(dtype).min
        x[:, 100:], z[:, 110:] = -inf, -inf
        ids[3] = 120                                        # no probability in the target, none in the draft
        ids[4] = 105                                        # none in the target alone
        x[8], z[6] = lowest, lowest                         # every column equal
        x[12, :64] = lowest
        x[16] = -inf                                        # request 4: no distribution at its first row
        x[21, 5] = float("nan")                             # request 5: at its second
        x[26, 7] = inf                                      # request 6: at its third
        z[21] = -inf                                        # request 7: a draft without a distribution
        z[24, 3], z[28, 1] = float("nan"), inf
        ids[30], ids[34] = -1, 130                          # no token
        for draft in (z, None):
            _check(mx, x, offsets, ids, u, noise, draft)


def test_noise_of_any_size(mx):
    x, offsets, ids, u, noise, z = _case([2] * 50, 90, torch.float32, 9)
    g = _gen(2)
    noise = noise * 2.0 ** torch.randint(-8, 9, noise.shape, generator=g, device="cuda")
    noise[3] = 2.0 ** -32
    noise[4] = 2.0 ** 32
    noise[5, :50], noise[5, 50:] = 2.0 ** -32, 2.0 ** 32
    _check(mx, x, offsets, ids, u, noise, z)
    noise[7, ::2] = -1.0                                    # not above 0: never drawn
    noise[8] = float("inf")
    noise[9, :80] = float("nan")
    r = _check(mx, x, offsets, ids, u, noise, z)
    at = int(offsets[8] + r.accepted[8])
    assert r.tokens[at] == -1 and bool(r.logprobs[at].isnan())


def test_strided_rows(mx):
    x, offsets, ids, u, noise, z = _case([2, 0, 3], 333, torch.bfloat16, 10)
    wide = torch.full((8, 400), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 7:340] = x
    wz = torch.full((5, 351), float("nan"), dtype=torch.bfloat16, device="cuda")
    wz[:, 3:336] = z
    wn = torch.full((3, 341), float("nan"), device="cuda")
    wn[:, 1:334] = noise
    _check(mx, wide[:, 7:340], offsets, ids, u, wn[:, 1:334], wz[:, 3:336])


def test_no_requests_and_malformed_offsets(mx):
    e = torch.empty
    r = mx.verify_drafts(e((0, 9), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"),
                         e(0, dtype=torch.long, device="cuda"), e(0, device="cuda"), e((0, 9), device="cuda"))
    assert r.accepted.numel() == r.tokens.numel() == 0
    x, offsets, ids, u, noise, z = _case([2, 3, 0, 1], 77, torch.float32, 11)
    good = mx.verify_drafts(x, torch.tensor(offsets, dtype=torch.int32, device="cuda"), ids, u, noise, draft_logits=z)
    for bad in ([0, 10, 0, 10, 0], [-5, 3, 3, 3, 99], [10, 8, 6, 4, 2], [0, 0, 0, 0, 0], [1 << 30, -(1 << 31), 5, 7, 2], [9, 10, 10, 10, 10]):
        r = mx.verify_drafts(x, torch.tensor(bad, dtype=torch.int32, device="cuda"), ids, u, noise, draft_logits=z)
        torch.cuda.synchronize()
        for b in range(4):
            if min(max(bad[b + 1], 0), 10) <= min(max(bad[b], 0), 10):
                assert r.accepted[b] == 0
    again = mx.verify_drafts(x, torch.tensor(offsets, dtype=torch.int32, device="cuda"), ids, u, noise, draft_logits=z)
    assert torch.equal(good.tokens, again.tokens) and torch.equal(good.logprobs, again.logprobs)


def test_streams_and_graphs(mx):
    a, b = (_case([3, 1, 0, 5], 5000, torch.bfloat16, s) for s in (20, 21))
    off = torch.tensor(a[1], dtype=torch.int32, device="cuda")

    def call(c):
        return mx.verify_drafts(c[0], off, c[2], c[3], c[4], draft_logits=c[5])
    want = [call(a), call(b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r = call(a)
    side.synchronize()
    assert torch.equal(r.tokens, want[0].tokens) and torch.equal(r.logprobs, want[0].logprobs)
    graphs = []
    for c in (a, b):
        inputs = [t.clone() if torch.is_tensor(t) else t for t in c]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(inputs)
        graphs.append((graph, inputs, out))
    for k, n in ((0, 0), (1, 1), (0, 1), (1, 0), (0, 0)):
        graph, inputs, out = graphs[k]
        for t, v in zip(inputs, (a, b)[n]):
            if torch.is_tensor(t):
                t.copy_(v)
        graph.replay()
        call((b, a)[n])
        torch.cuda.synchronize()
        assert torch.equal(out.accepted, want[n].accepted) and torch.equal(out.tokens, want[n].tokens)
        assert torch.equal(out.logprobs, want[n].logprobs)


def test_logits_past_the_caches(mx):
    """More than 96 MB of fp32 logits with rows at any 4 bytes, and of bf16 ones without a draft at any 2"""
    case = _case([5] * 36, 70001, torch.float32, 9)
    assert (case[0].numel() + case[5].numel()) * 4 > 96 << 20
    _check(mx, *case)
    case = _case([0, 5, 3, 7] * 30, 120001, torch.bfloat16, 10, draft=False)
    assert case[0].numel() * 2 > 96 << 20
    _check(mx, *case)
