"""The checkpoint, adapter and draft calls together: the example's learner and
sampler steps against full precision, also in captured graphs, and the expert
example with its activations kept in 8 bits."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16


def _example(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, "examples", name + ".py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _inputs(cfg, T, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((T, cfg.hidden), generator=g, device="cuda").to(BF16)
    policy = torch.randint(-1, cfg.policies, (T,), generator=g, device="cuda").to(torch.int32)
    targets = torch.randint(0, cfg.vocab, (T,), generator=g, device="cuda")
    targets[::7] = -1
    return x, policy, targets, torch.randn(T, generator=g, device="cuda")


def _cosine(a, b):
    return (torch.dot(a.double().flatten(), b.double().flatten()) / (a.double().norm() * b.double().norm())).item()


def test_learner_step_gradients(mx):
    """Cosine with fp32 autograd of the same weights.  An MXFP8 product of K terms of independent rounding (each factor
    off by at most 2^-4 of itself) is off by about 2^-4 sqrt(2/3) = 5% of its norm, a tensor kept in 8 bits by half of
    that; the longest path (gate_up's a) has three products forwards, two backwards and two kept tensors: 13%, a cosine
    of 0.99.  Twice that error would be 0.965."""
    ex = _example("adapter_policy_step")
    cfg = ex.Config(hidden=256, inter=384, vocab=640, rank=16, policies=5, scale=24.0)
    model = ex.AdapterPolicies(cfg, seed=3)
    T = 300
    x, policy, targets, adv = _inputs(cfg, T, 4)
    print("learner step", T, cfg, flush=True)
    got = model.backward(model.forward(x, policy), targets, adv)

    leaves = {n: [w.float().requires_grad_() for w in model.adapters[n]] for n in model.adapters}
    xf = x.float().requires_grad_()
    has = (policy >= 0).float().unsqueeze(1)
    at = policy.long().clamp_min(0)

    def project(name, v):
        a, b = leaves[name]
        hidden = (a[at] * v.unsqueeze(1)).sum(2)
        return v @ model.base[name].t() + has * model.scales[at].unsqueeze(1) * (b[at] * hidden.unsqueeze(1)).sum(2)
    gate, up = project("gate_up", xf).chunk(2, 1)
    out = xf + project("down", torch.nn.functional.silu(gate) * up)
    lp = torch.log_softmax(out @ model.base["head"].t(), 1).gather(1, targets.clamp_min(0).unsqueeze(1)).squeeze(1)
    loss = -(torch.where(targets >= 0, lp, 0.0) * adv).sum() / T
    loss.backward()
    assert _cosine(got["logprobs"], torch.where(targets >= 0, lp, 0.0).detach()) > 0.99
    for name in leaves:
        for i in range(2):
            assert _cosine(got[name][i], leaves[name][i].grad) > 0.965, (name, i)
    assert _cosine(got["x"], xf.grad) > 0.965


def _draft_inputs(cfg, B, n, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    offsets = torch.arange(0, B * (n + 1) + 1, n + 1, dtype=torch.int32, device="cuda")
    policy = torch.randint(-1, cfg.policies, (B,), generator=g, device="cuda").to(torch.int32).repeat_interleave(n + 1)
    x = torch.randn((B * (n + 1), cfg.hidden), generator=g, device="cuda").to(BF16)
    noise = torch.empty((B, cfg.vocab), device="cuda").exponential_(generator=g)
    return x, policy, offsets, torch.rand(B * n, generator=g, device="cuda"), noise, g


def test_sampler_step(mx):
    """A draft that is the model itself is always accepted; one of half its adapters sometimes; the tokens' scores are
    those of the target's own logits."""
    ex = _example("adapter_policy_step")
    cfg = ex.Config(hidden=256, inter=256, vocab=896, rank=8, policies=3, scale=60.0)
    model = ex.AdapterPolicies(cfg, seed=1)
    B, n = 20, 3
    x, policy, offsets, u, noise, g = _draft_inputs(cfg, B, n, 2)
    logits = model.forward(x, policy, keep=False)["logits"]
    drafted = torch.ones(B * (n + 1), dtype=torch.bool, device="cuda")
    drafted[n::n + 1] = False
    race = torch.empty((B * n, cfg.vocab), device="cuda").exponential_(generator=g)
    own = logits[drafted].contiguous()
    ids = torch.argmax(own.float() - torch.log(race), 1)
    v = model.verify(x, policy, offsets, ids, u, noise, draft_logits=own)
    assert bool((v.accepted == n).all()) and torch.equal(v.tokens[drafted], ids) and bool((v.tokens >= 0).all())
    assert torch.equal(model.forward(x, policy)["logits"], logits)                # keeping changes nothing
    # the base model alone as the draft
    base = model.forward(x, torch.full_like(policy, -1), keep=False)["logits"][drafted].contiguous()
    ids = torch.argmax(base.float() - torch.log(race), 1)
    v = model.verify(x, policy, offsets, ids, u, noise, draft_logits=base)
    total = int(v.accepted.sum())
    assert 0 < total < B * n
    scored = mx.token_logprobs(logits, v.tokens)
    real = v.tokens >= 0
    assert int(real.sum()) == total + B
    # both are log p of the same logits; their sums may differ by 2^-16 of them and a step of fp32
    assert bool(((v.logprobs - scored.logprobs).abs() <= 2.0 ** -15 + 2.0 ** -22 * scored.logprobs.abs())[real].all())


def test_steps_in_graphs(mx):
    """Both steps captured, replayed with other inputs between eager steps, each replay against the eager result."""
    ex = _example("adapter_policy_step")
    cfg = ex.Config(hidden=128, inter=128, vocab=384, rank=8, policies=3)
    model = ex.AdapterPolicies(cfg, seed=2)
    B, n = 6, 2
    data = []
    for seed in (1, 2):
        x, policy, offsets, u, noise, g = _draft_inputs(cfg, B, n, seed)
        ids = torch.randint(0, cfg.vocab, (B * n,), generator=g, device="cuda")
        data.append((x, policy, ids, u, noise, torch.randint(0, cfg.vocab, (B * (n + 1),), generator=g, device="cuda"),
                     torch.randn(B * (n + 1), generator=g, device="cuda")))

    def sampler(x, policy, ids, u, noise, targets, adv):
        v = model.verify(x, policy, offsets, ids, u, noise, temperature=0.8)
        return v.accepted, v.tokens, v.logprobs

    def learner(x, policy, ids, u, noise, targets, adv):
        r = model.backward(model.forward(x, policy), targets, adv)
        return (*r["gate_up"], *r["down"], r["x"], r["logprobs"])
    for step in (sampler, learner):
        want = [[t.clone() for t in step(*d)] for d in data]
        inputs = [t.clone() for t in data[0]]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(*inputs)
        for i in (1, 0, 0, 1):
            for t, v in zip(inputs, data[i]):
                t.copy_(v)
            graph.replay()
            step(*data[1 - i])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want[i])), (step.__name__, i)


def test_example_runs(mx, capsys):
    ex = _example("adapter_policy_step")
    import sys
    argv, sys.argv = sys.argv, ["adapter_policy_step.py", "--requests", "5", "--drafts", "2", "--steps", "2"]
    try:
        ex.main()
    finally:
        sys.argv = argv
    assert capsys.readouterr().out.count("step ") == 2


def test_expert_step_with_kept_activations(mx):
    """The expert example with gate | up kept in 8 bits and the product computed again: its gradients against those of
    the step that keeps both, off by the checkpoint's rounding (half of an MXFP8 product's 5%, once or twice)."""
    ex = _example("moe_policy_step")
    sizes = dict(hidden=256, inter=128, experts=16, k=3, vocab=640, groups=4, groups_kept=2, scale=1.5)
    T = 256
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    x = torch.randn((T, 256), generator=g, device="cuda").to(BF16)
    targets = torch.randint(0, 640, (T,), generator=g, device="cuda")
    adv = torch.randn(T, generator=g, device="cuda")
    grads = []
    for checkpoint in (False, True):
        model = ex.MoePolicy(ex.Config(**sizes, checkpoint=checkpoint), seed=5)
        s = model.forward(x, targets)
        assert ("gu" in s, "saved" in s) == (not checkpoint, checkpoint)
        grads.append((s["scored"].logprobs.clone(), model.backward(s, adv, 0.02)))
    # the forward pass rounds the product once to bf16 either way
    assert _cosine(grads[0][0], grads[1][0]) > 0.9999
    for name in ("router", "gate_up", "down", "head", "x"):
        assert _cosine(grads[0][1][name], grads[1][1][name]) > 0.99, name
