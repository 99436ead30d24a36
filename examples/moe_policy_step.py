"""One policy-gradient step of a mixture-of-experts layer and its LM head.

    python examples/moe_policy_step.py [--tokens 1024] [--steps 5]

The step a learner runs after sampling: the router picks the experts
(route, route_tables), the experts' GEMMs run in MXFP8 on rows sorted by
expert, moe_combine brings them back to token order, the head gives logits,
and token_logprobs scores the sampled tokens.  The loss is

    -(sum_t advantage_t log p(target_t) + beta entropy_t) / tokens

and its gradient goes the whole way back: token_logprobs_backward (in place
of the logits), the head, moe_combine_backward, both expert projections,
route_backward.  Nothing is copied to the host inside a step.
"""
import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_block_scaled_05_amd as mx  # noqa: E402

BF16 = torch.bfloat16


def _grid(batch, n, k, device):
    """Room for [batch][n][k] in the GEMMs' packed operand layout."""
    buffers = [torch.empty(mx.packed_bytes(batch, n, k, i), dtype=torch.uint8, device=device) for i in (0, 1)]
    return mx.PackedWeight(*buffers, batch, n, k)


def _token_grid(cols, rows, device):
    """A token-blocked grid [cols][rows], the weight gradients' operand."""
    return (torch.empty((cols, rows), dtype=torch.uint8, device=device),
            torch.empty((cols, rows // 32), dtype=torch.uint8, device=device))


@dataclass
class Config:
    """Sizes in multiples of 128; choice as mx.route takes it.  checkpoint: gate | up kept in 8 bits for the backward
    pass, which computes the experts' product again (2.06 bytes a value of it instead of 5.03)."""
    hidden: int = 1024
    inter: int = 512
    experts: int = 32
    k: int = 4
    vocab: int = 8192
    groups: int = 4
    groups_kept: int = 2
    scale: float = 1.0
    checkpoint: bool = False


class MoePolicy:
    def __init__(self, cfg: Config, device="cuda", seed: int = 0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def draw(*shape, std):
            return torch.randn(shape, generator=g, device=device) * std
        c, self.cfg, self.device = cfg, cfg, device
        self.router = draw(c.experts, c.hidden, std=c.hidden ** -0.5)
        self.balance = draw(c.experts, std=0.02)          # moved by the balancing rule of the trainer, not by gradients
        self.gate_up = draw(c.experts, 2 * c.inter, c.hidden, std=c.hidden ** -0.5)
        self.down = draw(c.experts, c.hidden, c.inter, std=c.inter ** -0.5)
        self.head = draw(c.vocab, c.hidden, std=c.hidden ** -0.5)
        self._grids = {}
        for name in ("gate_up", "down", "head"):
            w = getattr(self, name)
            batch, n, k = w.shape if w.dim() == 3 else (1, *w.shape)
            self._grids[name] = _grid(batch, n, k, device), _grid(batch, k, n, device)
        self.refresh()

    def choice(self):
        c = self.cfg
        return dict(score="sigmoid", bias=self.balance, groups=c.groups, groups_kept=c.groups_kept, group_top=2,
                    renormalize=True, scale=c.scale)

    def refresh(self):
        """The MXFP8 weights, blocked along K for the forward products and along N for the data gradients."""
        for name, (along_k, along_n) in self._grids.items():
            mx.quantize_dual_packed_(getattr(self, name).to(BF16), along_k, along_n)

    def forward(self, x: torch.Tensor, targets: torch.Tensor) -> dict:
        """x bf16 [T, hidden] (T a multiple of 128), targets int64 [T]."""
        c, dev, T = self.cfg, self.device, x.shape[0]
        s = {"x": x, "targets": targets}
        s["scores"] = x.float() @ self.router.t()
        s["ids"], s["w"] = mx.route(s["scores"], c.k, **self.choice())
        t = s["tables"] = mx.route_tables(s["ids"], c.experts, pad=32)
        rows = t.row_token.numel()
        # the weight gradients' grids start every expert on a multiple of 128 rows
        s["offsets128"] = mx.route_tables(s["ids"], c.experts, pad=128).offsets
        s["rows128"] = mx.route_rows(T * c.k, c.experts, 128)
        xq = _grid(1, rows, c.hidden, dev)
        mx.quantize_gather_packed_(x, t.row_token, xq)
        # rows after the last group are not written by the grouped GEMMs: they start as zeros
        gu = torch.zeros((rows, 2 * c.inter), dtype=BF16, device=dev)
        mx.grouped_gemm_packed(xq, self._grids["gate_up"][0], t.offsets, BF16, out=gu)
        if c.checkpoint:
            act = mx.swiglu(gu, layout="packed")
            h1, s["saved"] = act.h, (act.saved_q, act.saved_s)
        else:
            s["gu"] = gu
            gate, up = gu.float().chunk(2, 1)
            h = (torch.nn.functional.silu(gate) * up).to(BF16)
            s["h0"], h1 = _token_grid(c.inter, s["rows128"], dev), _grid(1, rows, c.inter, dev)
            mx.quantize_dual_grouped_packed_(h, t.offsets, s["offsets128"], s["h0"], h1)
        s["y"] = torch.zeros((rows, c.hidden), dtype=BF16, device=dev)
        mx.grouped_gemm_packed(h1, self._grids["down"][0], t.offsets, BF16, out=s["y"])
        hid = x + mx.moe_combine(s["y"], t.pair_row, s["w"])
        hid_row, s["hid_col"] = _grid(1, T, c.hidden, dev), _grid(1, c.hidden, T, dev)
        mx.quantize_dual_packed_(hid, hid_row, s["hid_col"])
        s["logits"] = mx.gemm_packed(hid_row, self._grids["head"][0], BF16)
        s["scored"] = mx.token_logprobs(s["logits"], targets)
        return s

    def backward(self, s: dict, advantage: torch.Tensor, beta: float) -> dict:
        """Gradients of the weights and of x; the logits in s are overwritten."""
        c, dev = self.cfg, self.device
        x, t, r = s["x"], s["tables"], s["scored"]
        T, rows = x.shape[0], t.row_token.numel()
        d_lp = -advantage / T
        d_entropy = torch.full_like(d_lp, -beta / T)
        d_logits = mx.token_logprobs_backward(s["logits"], s["targets"], r.stats, r.entropy, d_lp, d_entropy,
                                              out=s["logits"])
        dl_row, dl_col = _grid(1, T, c.vocab, dev), _grid(1, c.vocab, T, dev)
        mx.quantize_dual_packed_(d_logits, dl_row, dl_col)
        d_hid = mx.gemm_packed(dl_row, self._grids["head"][1], BF16)
        out = {"head": mx.gemm_packed(dl_col, s["hid_col"], torch.float32)}

        d_y, d_w = mx.moe_combine_backward(d_hid, s["y"], t.pair_row, s["w"], t.row_token)
        dy0, dy1 = _token_grid(c.hidden, s["rows128"], dev), _grid(1, rows, c.hidden, dev)
        mx.quantize_dual_grouped_packed_(d_y, t.offsets, s["offsets128"], dy0, dy1)
        d_h = torch.zeros((rows, c.inter), dtype=BF16, device=dev)
        mx.grouped_gemm_packed(dy1, self._grids["down"][1], t.offsets, BF16, out=d_h)
        if c.checkpoint:
            d_gu, h = mx.swiglu_backward(d_h, *s["saved"])
            h0 = _token_grid(c.inter, s["rows128"], dev)
            mx.quantize_dual_grouped_into(h, t.offsets, s["offsets128"], *h0)
        else:
            h0 = s["h0"]
            gate, up = s["gu"].float().chunk(2, 1)
            sig = torch.sigmoid(gate)
            d_gate = d_h.float() * up * sig * (1 + gate * (1 - sig))
            d_gu = torch.cat((d_gate, d_h.float() * gate * sig), 1).to(BF16)
        out["down"] = mx.grouped_gemm_wgrad(*dy0, *h0, s["offsets128"], torch.float32)

        dg0, dg1 = _token_grid(2 * c.inter, s["rows128"], dev), _grid(1, rows, 2 * c.inter, dev)
        mx.quantize_dual_grouped_packed_(d_gu, t.offsets, s["offsets128"], dg0, dg1)
        d_rows = torch.zeros((rows, c.hidden), dtype=BF16, device=dev)
        mx.grouped_gemm_packed(dg1, self._grids["gate_up"][1], t.offsets, BF16, out=d_rows)
        sorted_x = torch.where(t.row_token.unsqueeze(1) >= 0, x[t.row_token.clamp_min(0)], 0)
        x0 = _token_grid(c.hidden, s["rows128"], dev)
        mx.quantize_dual_grouped_into(sorted_x, t.offsets, s["offsets128"], *x0)
        out["gate_up"] = mx.grouped_gemm_wgrad(*dg0, *x0, s["offsets128"], torch.float32)

        kw = self.choice()
        d_scores = mx.route_backward(s["scores"], s["ids"], d_w, score=kw["score"], renormalize=kw["renormalize"],
                                     scale=kw["scale"])
        out["router"] = d_scores.t() @ x.float()
        # a token's gradient: its residual, its experts' rows, its router scores
        out["x"] = d_hid.float() + d_scores @ self.router + mx.moe_combine(d_rows, t.pair_row,
                                                                          torch.ones_like(s["w"])).float()
        return out

    def step(self, x, targets, advantage, beta: float = 0.0, lr: float = 0.1):
        """One update by gradient descent.  Returns the scored tokens (TokenLogprobs)."""
        s = self.forward(x, targets)
        grads = self.backward(s, advantage, beta)
        for name in ("router", "gate_up", "down", "head"):
            getattr(self, name).sub_(lr * grads[name])
        self.refresh()
        return s["scored"]


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=1024)
    p.add_argument("--steps", type=int, default=5)
    a = p.parse_args()
    cfg = Config()
    model = MoePolicy(cfg)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((a.tokens, cfg.hidden), generator=g, device="cuda").to(BF16)
    targets = torch.randint(0, cfg.vocab, (a.tokens,), generator=g, device="cuda")
    advantage = torch.ones(a.tokens, device="cuda")
    for i in range(a.steps):
        r = model.step(x, targets, advantage, beta=0.001, lr=2.0)
        print("step %d: mean log-probability %.4f, mean entropy %.4f" % (i, r.logprobs.mean().item(), r.entropy.mean().item()),
              flush=True)


if __name__ == "__main__":
    main()
