"""The routing, combine and log-probability calls together: the example's
learner step against full-precision autograd, and the calls in a captured
graph."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("moe_policy_step", os.path.join(ROOT, "examples", "moe_policy_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _inputs(cfg, T, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((T, cfg.hidden), generator=g, device="cuda").to(torch.bfloat16)
    targets = torch.randint(0, cfg.vocab, (T,), generator=g, device="cuda")
    targets[::9] = -100
    return x, targets, torch.randn(T, generator=g, device="cuda")


def test_learner_step_gradients(mx):
    """Cosine with fp32 autograd of the same weights and the same choice.  An
    MXFP8 product of K terms of independent rounding (each factor off by at
    most 2^-4 of itself) is off by about 2^-4 sqrt(2/3) = 5% of its norm, and
    the longest path has seven of them in a row: 14%, a cosine of 0.99."""
    import torch
    ex = _example()
    cfg = ex.Config(hidden=256, inter=128, experts=16, k=3, vocab=640, groups=4, groups_kept=2, scale=1.5)
    model = ex.MoePolicy(cfg, seed=5)
    T, beta = 256, 0.02
    x, targets, adv = _inputs(cfg, T, 6)
    print("learner step", T, cfg, flush=True)
    s = model.forward(x, targets)
    logp, entropy = s["scored"].logprobs.clone(), s["scored"].entropy.clone()
    got = model.backward(s, adv, beta)

    leaves = {n: getattr(model, n).clone().requires_grad_() for n in ("router", "gate_up", "down", "head")}
    xf = x.float().requires_grad_()
    sc = torch.sigmoid(xf @ leaves["router"].t())
    a = sc.gather(1, s["ids"].long())
    w = a / a.sum(1, keepdim=True) * cfg.scale
    out = xf
    for j in range(cfg.k):
        e = s["ids"][:, j].long()
        gu = (leaves["gate_up"][e] * xf.unsqueeze(1)).sum(2)
        h = torch.nn.functional.silu(gu[:, :cfg.inter]) * gu[:, cfg.inter:]
        out = out + w[:, j:j + 1] * (leaves["down"][e] * h.unsqueeze(1)).sum(2)
    lp = torch.log_softmax(out @ leaves["head"].t(), 1)
    H = -(lp.exp() * lp).sum(1)
    real = targets >= 0
    chosen = torch.where(real, lp.gather(1, targets.clamp_min(0).unsqueeze(1)).squeeze(1), 0.0)
    (-(adv * chosen + beta * H).sum() / T).backward()
    cos = torch.nn.functional.cosine_similarity
    assert cos(logp[real], chosen[real].detach(), 0) > 0.99 and cos(entropy, H.detach(), 0) > 0.99
    assert torch.all(logp[~real] == 0)
    for n, leaf in list(leaves.items()) + [("x", xf)]:
        c = cos(got[n].flatten().float(), leaf.grad.flatten(), 0).item()
        assert c > 0.95, (n, c)


def test_learner_steps_raise_the_rewarded_tokens(mx):
    import torch
    ex = _example()
    cfg = ex.Config(hidden=256, inter=128, experts=16, k=3, vocab=640)
    model = ex.MoePolicy(cfg, seed=7)
    x, targets, _ = _inputs(cfg, 256, 8)
    means = []
    for _ in range(4):
        means.append(model.step(x, targets, torch.ones(256, device="cuda"), lr=5.0).logprobs.mean().item())
    assert all(b > a for a, b in zip(means, means[1:])), means


@pytest.mark.parametrize("T", [1, 700])
def test_token_calls_in_a_graph(mx, T):
    """Every replay gives the bits of the eager calls on the inputs of the moment."""
    import torch
    E, k, H, V = 64, 6, 200, 40000
    print("graph", T, flush=True)
    scores = torch.zeros((T, E), device="cuda")
    rows = mx.route_rows(T * k, E, 32)
    y = torch.zeros((rows, H), device="cuda", dtype=torch.bfloat16)
    d_out = torch.zeros((T, H), device="cuda", dtype=torch.bfloat16)
    logits = torch.zeros((T, V), device="cuda", dtype=torch.bfloat16)
    targets = torch.zeros(T, dtype=torch.int64, device="cuda")
    grad = torch.zeros(T, device="cuda")
    kw = dict(score="sigmoid", renormalize=True, scale=2.0)

    def chain():
        ids, w = mx.route(scores, k, groups=8, groups_kept=4, **kw)
        t = mx.route_tables(ids, E)
        out = mx.moe_combine(y, t.pair_row, w)
        d_y, d_w = mx.moe_combine_backward(d_out, y, t.pair_row, w, t.row_token)
        d_scores = mx.route_backward(scores, ids, d_w, **kw)
        r = mx.token_logprobs(logits, targets, top_n=5)
        d_logits = mx.token_logprobs_backward(logits, targets, r.stats, r.entropy, grad, grad)
        return (ids, w, t.offsets, t.counts, t.row_token, t.pair_row, out, d_y, d_w, d_scores, r.logprobs, r.entropy,
                r.stats, r.top_logprobs, r.top_ids, d_logits)

    def fill(seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        for z in (scores, y, d_out, logits, grad):
            z.copy_(torch.randn(z.shape, generator=g, device="cuda"))
        targets.copy_(torch.randint(-1, V, (T,), generator=g, device="cuda"))

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = chain()
    for seed in range(1, 5):
        fill(seed)
        want = [z.clone() for z in chain()]
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(captured, want)):
            assert torch.equal(a, b), (seed, i)
