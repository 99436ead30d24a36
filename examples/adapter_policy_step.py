"""Policies of one base model, each with its own low-rank adapters: a step of the
sampler that verifies drafted tokens, and a step of the learner.

    python examples/adapter_policy_step.py [--requests 24] [--drafts 4] [--steps 3]

The base weights (an MLP block and the head) stay in MXFP8 as the GEMMs read
them; what is trained is the adapters, several policies in one batch.

Sampler: the drafted positions of all requests run through the block (shared
GEMMs, each request's adapters beside them) to the target's logits, and
verify_drafts takes the tokens that stand and the one after them.

Learner: the same block over the sampled rows.  What the backward pass needs is
kept in 8 bits: the GEMM operands themselves as the adapters' inputs, and gate |
up as swiglu's checkpoint.  The loss is  -sum_t advantage_t log p(target_t) / rows.
Nothing is copied to the host inside a step.
"""
import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_block_scaled_05_amd as mx  # noqa: E402

BF16 = torch.bfloat16


def _grid(n, k, device):
    """Room for [n][k] in the GEMMs' packed operand layout."""
    return mx.PackedWeight(*(torch.empty(mx.packed_bytes(1, n, k, i), dtype=torch.uint8, device=device) for i in (0, 1)), 1, n, k)


@dataclass
class Config:
    """Sizes in multiples of 128; adapters of `rank` (a multiple of 8) for each of `policies`."""
    hidden: int = 1024
    inter: int = 2048
    vocab: int = 8192
    rank: int = 16
    policies: int = 8
    scale: float = 2.0


class AdapterPolicies:
    def __init__(self, cfg: Config, device="cuda", seed: int = 0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def draw(*shape, std):
            return torch.randn(shape, generator=g, device=device) * std
        c, self.cfg, self.device = cfg, cfg, device
        self.base = {"gate_up": draw(2 * c.inter, c.hidden, std=c.hidden ** -0.5), "down": draw(c.hidden, c.inter, std=c.inter ** -0.5),
                     "head": draw(c.vocab, c.hidden, std=c.hidden ** -0.5)}
        # along K for the forward products, along N for the data gradients
        self.grids = {}
        for name, w in self.base.items():
            self.grids[name] = _grid(*w.shape, device), _grid(*reversed(w.shape), device)
            mx.quantize_dual_packed_(w.to(BF16), *self.grids[name])
        self.scales = torch.full((c.policies,), c.scale / c.rank, device=device)
        self.adapters = {}
        for name in ("gate_up", "down"):
            n, k = self.base[name].shape
            self.adapters[name] = [draw(c.policies, c.rank, k, std=k ** -0.5).to(BF16), draw(c.policies, n, c.rank, std=0.1).to(BF16)]

    def tables(self, policy: torch.Tensor):
        """Rows of every policy together: policy int32 [T] (outside [0, policies): the base model alone)."""
        return mx.route_tables(policy.view(-1, 1), self.cfg.policies)

    def _project(self, name, x, tables, keep):
        """(y, x as the GEMM's operand, hidden rows of the adapters)"""
        xq = _grid(*x.shape, self.device)
        mx.quantize_many_layouts_([(x, xq)])
        y = mx.gemm_packed(xq, self.grids[name][0], BF16)
        hidden = mx.lora_add_(y, x, *self.adapters[name], tables, self.scales, keep_hidden=keep)
        return y, xq, hidden

    def forward(self, x: torch.Tensor, policy: torch.Tensor, keep: bool = True) -> dict:
        """x bf16 [T, hidden] -> logits bf16 [T, vocab], and with ``keep`` what backward needs."""
        t = self.tables(policy)
        gu, xq, h1 = self._project("gate_up", x, t, keep)
        act = mx.swiglu(gu, save=keep)
        y, hq, h2 = self._project("down", act.h, t, keep)
        out = x + y
        oq = _grid(*out.shape, self.device)
        mx.quantize_many_layouts_([(out, oq)])
        s = {"logits": mx.gemm_packed(oq, self.grids["head"][0], BF16)}
        if keep:
            s.update(tables=t, xq=xq, hq=hq, h1=h1, h2=h2, saved=(act.saved_q, act.saved_s))
        return s

    def _back(self, name, d_y, xq, hidden, tables):
        """(gradient of the projection's input, of a, of b)"""
        dq = _grid(*d_y.shape, self.device)
        mx.quantize_many_layouts_([(d_y, dq)])
        d_x = mx.gemm_packed(dq, self.grids[name][1], BF16)
        return (d_x, *mx.lora_backward_(d_x, d_y, xq, *self.adapters[name], hidden, tables, self.scales))

    def backward(self, s: dict, targets: torch.Tensor, advantage: torch.Tensor) -> dict:
        """Gradients of the adapters and of x; the logits in s are overwritten."""
        T = targets.numel()
        r = mx.token_logprobs(s["logits"], targets)
        d_logits = mx.token_logprobs_backward(s["logits"], targets, r.stats, None, -advantage / T, out=s["logits"])
        dq = _grid(*d_logits.shape, self.device)
        mx.quantize_many_layouts_([(d_logits, dq)])
        d_out = mx.gemm_packed(dq, self.grids["head"][1], BF16)
        d_h, down_a, down_b = self._back("down", d_out, s["hq"], s["h2"], s["tables"])
        d_gu, _ = mx.swiglu_backward(d_h, *s["saved"], recompute=False)
        d_x, up_a, up_b = self._back("gate_up", d_gu, s["xq"], s["h1"], s["tables"])
        return {"gate_up": (up_a, up_b), "down": (down_a, down_b), "x": d_out.float() + d_x.float(), "logprobs": r.logprobs}

    def verify(self, x, policy, offsets, draft_ids, uniforms, noise, *, draft_logits=None, temperature=1.0):
        """The sampler's step: rows of x as verify_drafts wants the logits."""
        logits = self.forward(x, policy, keep=False)["logits"]
        return mx.verify_drafts(logits, offsets, draft_ids, uniforms, noise, draft_logits=draft_logits, temperature=temperature)

    def step(self, x, policy, targets, advantage, lr: float = 0.1):
        """One update of the adapters by gradient descent.  Returns the scored tokens' log-probabilities."""
        g = self.backward(self.forward(x, policy), targets, advantage)
        for name in ("gate_up", "down"):
            for w, d in zip(self.adapters[name], g[name]):
                w.copy_((w.float() - lr * d).to(BF16))
        return g["logprobs"]


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--requests", type=int, default=24)
    p.add_argument("--drafts", type=int, default=4)
    p.add_argument("--steps", type=int, default=3)
    a = p.parse_args()
    cfg = Config()
    model = AdapterPolicies(cfg)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    B, n = a.requests, a.drafts
    offsets = torch.arange(0, B * (n + 1) + 1, n + 1, dtype=torch.int32, device="cuda")
    policy = torch.randint(-1, cfg.policies, (B,), generator=g, device="cuda").to(torch.int32).repeat_interleave(n + 1)
    x = torch.randn((B * (n + 1), cfg.hidden), generator=g, device="cuda").to(BF16)
    for i in range(a.steps):
        ids = torch.randint(0, cfg.vocab, (B * n,), generator=g, device="cuda")
        u = torch.rand(B * n, generator=g, device="cuda")
        noise = torch.empty((B, cfg.vocab), device="cuda").exponential_(generator=g)
        v = model.verify(x, policy, offsets, ids, u, noise)
        lp = model.step(x, policy, v.tokens, torch.ones(v.tokens.numel(), device="cuda"), lr=20.0)
        print("step %d: %d drafted tokens stand, %d tokens, mean log-probability %.4f" % (
            i, v.accepted.sum().item(), (v.tokens >= 0).sum().item(), lp[v.tokens >= 0].mean().item()), flush=True)


if __name__ == "__main__":
    main()
