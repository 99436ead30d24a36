"""The measured cases of the router, expert-combine and token log-probability
operators, with their plain forms.

``run`` computes an operator either in its plain form (elementary torch
operations in fp32, fp64 where a comparison decides) or, with ``own`` true,
through this package's calls.  ``exact`` gives the same outputs in fp64 from
the definitions.

Operators (``case["op"]``):
  route          router logits -> expert ids and weights of every token
  route_grad     gradient of those weights -> gradient of the logits
  dispatch       expert ids -> the padded, expert-sorted row tables that the
                 grouped GEMMs and their quantizers read
  combine        weighted sum of a token's expert rows, back in token order
  combine_grad   its gradients (expert rows and weights)
  logprobs       log probability of given tokens, entropy, top alternatives
  logprobs_grad  gradient of log probability and entropy -> logits
"""
import math

import numpy as np
import torch

own = False

PAD = 32                 # rows of an expert's group are padded to this multiple
IGNORED = -100           # target of a position that has none (prompt tokens)

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_ESIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one token of a serving step through a 128-expert router: pure latency
        dict(name="route_token", op="route", T=1, E=128, k=8, dtype="f32", score="softmax", bias=False,
             groups=1, kept=1, group_top=1, renorm=True, scale=1.0),
        # a training micro-batch, sigmoid scores balanced by a bias, experts limited to 4 of 8 groups
        dict(name="route_groups", op="route", T=16384, E=256, k=8, dtype="f32", score="sigmoid", bias=True,
             groups=8, kept=4, group_top=2, renorm=True, scale=2.5),
        # the router's gradient over an odd number of tokens, plain softmax weights, bf16 logits
        dict(name="route_grad", op="route_grad", T=8191, E=128, k=8, dtype="bf16", score="softmax", bias=False,
             groups=1, kept=1, group_top=1, renorm=False, scale=1.0),
        # the tables of a small serving batch: pure latency
        dict(name="dispatch_serve", op="dispatch", T=32, E=128, k=8),
        # the tables of a training micro-batch
        dict(name="dispatch_train", op="dispatch", T=16384, E=256, k=8),
        # the expert outputs of a small serving batch
        dict(name="combine_serve", op="combine", T=16, E=128, k=8, H=2048, dtype="bf16"),
        # the expert outputs of a training micro-batch
        dict(name="combine_train", op="combine", T=8192, E=128, k=8, H=2048, dtype="bf16"),
        # their gradients, odd number of tokens
        dict(name="combine_grad", op="combine_grad", T=4095, E=128, k=8, H=2048, dtype="bf16"),
        # one answered token with its 20 best alternatives
        dict(name="logprobs_token", op="logprobs", T=1, V=131072, dtype="bf16", top=20, temperature=1.0),
        # the old-policy stage of a training step: log probability and entropy of every position, no gradient
        dict(name="logprobs_score", op="logprobs", T=2048, V=131072, dtype="bf16", top=0, temperature=1.0),
        # sampled positions with alternatives: fp32 logits, odd vocabulary, temperature
        dict(name="logprobs_top", op="logprobs", T=511, V=100003, dtype="f32", top=5, temperature=0.7),
        # the gradient of the policy loss with an entropy term
        dict(name="logprobs_grad", op="logprobs_grad", T=2048, V=131072, dtype="bf16", temperature=1.0),
    ]


def _log_int(rng, lo, hi):
    # spread over the logarithm; whole multiples of 1024 are left to the listed cases
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n if n % 1024 else n - 1


def draw(rng):
    op = rng.choice(["route", "route_grad", "dispatch", "combine", "combine_grad", "logprobs", "logprobs_grad"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8])
        size = _log_int(rng, 8, 512 // groups if groups > 1 else 512)
        E = groups * size
        kept = rng.randint(1, groups)
        k = rng.randint(1, min(10, kept * size))
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=k, dtype=dtype, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, kept=kept, group_top=rng.choice([1, 2]),
                    renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]))
    E = _log_int(rng, 8, 512)
    k = rng.randint(1, min(10, E))
    if op == "dispatch":
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=k)
    if op in ("combine", "combine_grad"):
        H = _log_int(rng, 64, 4096)
        if rng.random() < 0.6:
            H = H // 16 * 16 + 8
        most = max(1, (1 << 26) // (k * H))              # at most 2^26 expert values
        return dict(op=op, T=_log_int(rng, 1, min(8192, most)), E=E, k=k, H=H, dtype=dtype)
    V = _log_int(rng, 1000, 131072)
    T = _log_int(rng, 1, min(8192, (1 << 27) // V))
    case = dict(op=op, T=T, V=V, dtype=dtype, temperature=rng.choice([1.0, 0.7, 1.3]))
    if op == "logprobs":
        case["top"] = rng.choice([0, 1, 5, 20])
    return case


def _rows(T, k, E):
    """Rows that the padded groups of T*k pairs over E experts can take at most."""
    pairs = T * k
    return (pairs + min(E, pairs) * (PAD - 1)) // PAD * PAD


def work(case):
    op, T = case["op"], case["T"]
    if op in ("logprobs", "logprobs_grad"):
        n = T * case["V"]
        e = _ESIZE[case["dtype"]]
        if op == "logprobs":                             # scale, exp, two sums, maximum
            return {"bytes": n * e + T * 8 + T * 8 + T * case["top"] * 12, "flops": 6 * n}
        return {"bytes": 2 * n * e + T * 8 + T * 20, "flops": 8 * n}
    k, E = case["k"], case["E"]
    pairs = T * k
    if op == "route":
        return {"bytes": T * E * _ESIZE[case["dtype"]] + (E * 4 if case["bias"] else 0) + pairs * 8,
                "flops": 6 * T * E}
    if op == "route_grad":
        return {"bytes": 2 * T * E * _ESIZE[case["dtype"]] + pairs * 8, "flops": 6 * T * E}
    if op == "dispatch":
        return {"bytes": pairs * 8 + _rows(T, k, E) * 8 + (2 * E + 1) * 4, "flops": pairs}
    H, e = case["H"], _ESIZE[case["dtype"]]
    if op == "combine":
        return {"bytes": pairs * H * e + T * H * e + pairs * 8, "flops": 2 * pairs * H}
    return {"bytes": pairs * H * e + T * H * e + _rows(T, k, E) * (H * e + 8) + pairs * 12, "flops": 3 * pairs * H}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _router_logits(case, g):
    # a common preference for some experts and a token's own choice
    T, E = case["T"], case["E"]
    x = torch.randn((T, E), generator=g, device="cuda") * 1.2
    x += torch.randn((1, E), generator=g, device="cuda") * 0.6
    return x.to(_TYPES[case["dtype"]])


def _skewed_ids(T, E, k, g):
    # distinct experts of each token, popularity falling as 1/rank^1.1
    p = -1.1 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    u = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    return torch.topk(p - torch.log(-torch.log(u)), k, dim=1).indices.to(torch.int32)


def prepare(case, seed):
    g = _generator(seed)
    op, T = case["op"], case["T"]
    st = dict(case)
    if op in ("route", "route_grad"):
        st["logits"] = _router_logits(case, g)
        st["bias"] = (torch.randn(case["E"], generator=g, device="cuda") * 0.05) if case["bias"] else None
        if op == "route_grad":
            st["ids"] = _plain_route(st)[0]
            st["d_weights"] = torch.randn((T, case["k"]), generator=g, device="cuda") * 2.0 ** -6
        return st
    if op == "dispatch":
        st["ids"] = _skewed_ids(T, case["E"], case["k"], g)
        return st
    if op in ("combine", "combine_grad"):
        t, rows = _TYPES[case["dtype"]], _rows(T, case["k"], case["E"])
        _, _, st["row_token"], st["pair_row"] = _plain_dispatch(_skewed_ids(T, case["E"], case["k"], g), case["E"])
        st["y"] = torch.randn((rows, case["H"]), generator=g, device="cuda").to(t)
        st["weights"] = torch.softmax(torch.randn((T, case["k"]), generator=g, device="cuda"), 1)
        if op == "combine_grad":
            st["d_out"] = (torch.randn((T, case["H"]), generator=g, device="cuda") * 2.0 ** -8).to(t)
        return st
    V = case["V"]
    x = torch.randn((T, V), generator=g, device="cuda") * 2.0
    # a few likely continuations stand out at every position (distinct ids: one in each 24th of those in use)
    used = V - V // 1024
    part = used // 24
    likely = torch.randint(0, part, (T, 24), generator=g, device="cuda") + part * torch.arange(24, device="cuda")
    x.scatter_(1, likely, 4.0 + 9.0 * torch.rand((T, 24), generator=g, device="cuda"))
    x[:, used:] = -math.inf                              # ids that the tokenizer does not use
    st["logits"] = x.to(_TYPES[case["dtype"]])
    # sampled continuations, now and then an unlikely one, and prompt positions without a target
    target = likely.gather(1, torch.randint(0, 24, (T, 1), generator=g, device="cuda")).squeeze(1)
    u = torch.rand((T,), generator=g, device="cuda")
    anywhere = torch.randint(0, used, (T,), generator=g, device="cuda")
    target = torch.where(u < 0.25, anywhere, target)
    st["targets"] = torch.where(u > 0.95, torch.full_like(target, IGNORED), target)
    if op == "logprobs_grad":
        _, st["entropy"], st["stats"] = _plain_logprobs(st)
        st["d_logprobs"] = torch.randn((T,), generator=g, device="cuda")
        st["d_entropy"] = torch.randn((T,), generator=g, device="cuda") * 2.0 ** -6
    return st


# ------------------------------------------------------------------ plain forms

def _plain_scores(st, wide):
    x = st["logits"].to(wide)
    if st["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.max(1, keepdim=True).values)
    return e / e.sum(1, keepdim=True)


def _plain_weights(s, st):
    w = s / s.sum(1, keepdim=True) if st["renorm"] else s
    return w * st["scale"]


def _plain_route(st):
    # the choice in fp64: two experts whose scores differ below fp32's step still have an order
    s = _plain_scores(st, torch.float64)
    c = s if st["bias"] is None else s + st["bias"].double()
    T, E = c.shape
    if st["groups"] > 1:
        size = E // st["groups"]
        best = torch.sort(c.view(T, st["groups"], size), dim=2, descending=True, stable=True).values
        score = best[:, :, :st["group_top"]].sum(2)
        kept = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :st["kept"]]
        keep = torch.zeros((T, st["groups"]), dtype=torch.bool, device=c.device)
        keep.scatter_(1, kept, True)
        c = torch.where(keep.repeat_interleave(size, 1), c, -math.inf)
    ids = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :st["k"]]
    chosen = torch.gather(s, 1, ids).float()
    return ids.to(torch.int32), _plain_weights(chosen, st)


def _plain_route_grad(st):
    s = _plain_scores(st, torch.float32)
    ids, dw = st["ids"].long(), st["d_weights"]
    chosen = torch.gather(s, 1, ids)
    ds = dw * st["scale"]
    if st["renorm"]:
        total = chosen.sum(1, keepdim=True)
        ds = (ds - (ds * chosen).sum(1, keepdim=True) / total) / total
    full = torch.zeros_like(s).scatter_(1, ids, ds)
    if st["score"] == "sigmoid":
        d = full * s * (1 - s)
    else:
        d = s * (full - (ds * chosen).sum(1, keepdim=True))
    return d.to(st["logits"].dtype)


def _plain_dispatch(ids, E):
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    pairs, rows = T * k, _rows(T, k, E)
    counts = torch.zeros(E, dtype=torch.long, device=ids.device).scatter_add_(0, flat, torch.ones_like(flat))
    padded = (counts + PAD - 1) // PAD * PAD
    offsets = torch.zeros(E + 1, dtype=torch.long, device=ids.device)
    offsets[1:] = torch.cumsum(padded, 0)
    first = torch.cumsum(counts, 0) - counts
    order = torch.sort(flat, stable=True).indices
    expert = flat[order]
    row = offsets[expert] + torch.arange(pairs, device=ids.device) - first[expert]
    pair_row = torch.zeros_like(flat).scatter_(0, order, row)
    row_token = torch.full((rows,), -1, dtype=torch.long, device=ids.device).scatter_(0, row, order // k)
    return (offsets.to(torch.int32), counts.to(torch.int32), row_token, pair_row.view(T, k).to(torch.int32))


def _plain_combine(st):
    y = st["y"][st["pair_row"].long()].float()
    return (y * st["weights"].unsqueeze(2)).sum(1).to(st["y"].dtype)


def _plain_combine_grad(st):
    row, d = st["pair_row"].long(), st["d_out"].float()
    d_weights = (st["y"][row].float() * d.unsqueeze(1)).sum(2)
    d_rows = (st["weights"].unsqueeze(2) * d.unsqueeze(1)).to(st["y"].dtype)
    d_y = torch.zeros_like(st["y"])
    d_y[row.view(-1)] = d_rows.view(-1, d.shape[1])
    return d_y, d_weights


def _plain_logprobs(st):
    z = st["logits"].float() / st["temperature"]
    m = z.max(1).values
    e = torch.exp(z - m.unsqueeze(1))
    total = e.sum(1)
    log_total = torch.log(total)
    weighted = torch.where(e > 0, e * (z - m.unsqueeze(1)), 0.0).sum(1)
    entropy = log_total - weighted / total
    t = st["targets"]
    zt = torch.gather(z, 1, t.clamp_min(0).unsqueeze(1)).squeeze(1)
    logprobs = torch.where(t >= 0, zt - m - log_total, 0.0)
    stats = torch.stack((m, log_total), 1)
    if not st.get("top"):
        return logprobs, entropy, stats
    best = torch.sort(st["logits"], dim=1, descending=True, stable=True)
    ids = best.indices[:, :st["top"]].contiguous()
    top = torch.gather(z, 1, ids) - m.unsqueeze(1) - log_total.unsqueeze(1)
    return logprobs, entropy, stats, top, ids


def _plain_logprobs_grad(st):
    z = st["logits"].float() / st["temperature"]
    logp = z - st["stats"][:, :1] - st["stats"][:, 1:]
    p = torch.exp(logp)
    t, g = st["targets"], st["d_logprobs"].unsqueeze(1)
    g = torch.where(t.unsqueeze(1) >= 0, g, 0.0)
    d = -g * p - torch.where(p > 0, st["d_entropy"].unsqueeze(1) * p * (logp + st["entropy"].unsqueeze(1)), 0.0)
    d.scatter_add_(1, t.clamp_min(0).unsqueeze(1), g)
    return (d / st["temperature"]).to(st["logits"].dtype)


# ------------------------------------------------------------------ one pass

def _run_own(st):
    import mxfp8_block_scaled_05_amd as mx
    op = st["op"]
    if op == "route":
        return mx.route(st["logits"], st["k"], score=st["score"], bias=st["bias"], groups=st["groups"],
                        groups_kept=st["kept"], group_top=st["group_top"], renormalize=st["renorm"], scale=st["scale"])
    if op == "route_grad":
        return mx.route_backward(st["logits"], st["ids"], st["d_weights"], score=st["score"],
                                 renormalize=st["renorm"], scale=st["scale"])
    if op == "dispatch":
        t = mx.route_tables(st["ids"], st["E"], pad=PAD)
        return t.offsets, t.counts, t.row_token, t.pair_row
    if op == "combine":
        return mx.moe_combine(st["y"], st["pair_row"], st["weights"])
    if op == "combine_grad":
        return mx.moe_combine_backward(st["d_out"], st["y"], st["pair_row"], st["weights"], st["row_token"])
    if op == "logprobs":
        r = mx.token_logprobs(st["logits"], st["targets"], temperature=st["temperature"], top_n=st["top"])
        out = (r.logprobs, r.entropy, r.stats)
        return out + (r.top_logprobs, r.top_ids) if st["top"] else out
    return mx.token_logprobs_backward(st["logits"], st["targets"], st["stats"], st["entropy"], st["d_logprobs"],
                                      st["d_entropy"], temperature=st["temperature"])


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "route":
        return _plain_route(state)
    if op == "route_grad":
        return _plain_route_grad(state)
    if op == "dispatch":
        return _plain_dispatch(state["ids"], state["E"])
    if op == "combine":
        return _plain_combine(state)
    if op == "combine_grad":
        return _plain_combine_grad(state)
    if op == "logprobs":
        return _plain_logprobs(state)
    return _plain_logprobs_grad(state)


# ------------------------------------------------------------------ fp64 definitions

def _np64(t):
    return t.double().cpu().numpy()


def _exact_route(st):
    x = _np64(st["logits"])
    T, E = x.shape
    if st["score"] == "softmax":
        s = np.exp(x - x.max(1)[:, None])
        s = s / s.sum(1)[:, None]
    else:
        s = np.reciprocal(1.0 + np.exp(-x))
    c = s.copy() if st["bias"] is None else s + _np64(st["bias"])[None]
    G = st["groups"]
    if G > 1:
        blocks = np.sort(c.reshape(T, G, E // G), axis=2)[:, :, ::-1]
        rank = np.argsort(-blocks[:, :, :st["group_top"]].sum(2), axis=1, kind="stable")
        closed = np.ones((T, G), bool)
        np.put_along_axis(closed, rank[:, :st["kept"]], False, axis=1)
        c[np.repeat(closed, E // G, axis=1)] = -np.inf
    ids = np.argsort(-c, axis=1, kind="stable")[:, :st["k"]]
    w = np.take_along_axis(s, ids, 1)
    if st["renorm"]:
        w = w / w.sum(1)[:, None]
    return torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(w * st["scale"]).cuda()


def _exact_route_grad(st):
    x, ids = _np64(st["logits"]), st["ids"].long().cpu().numpy()
    g = _np64(st["d_weights"]) * st["scale"]
    rows = np.arange(x.shape[0])[:, None]
    if st["score"] == "softmax":
        s = np.exp(x - x.max(1)[:, None])
        s = s / s.sum(1)[:, None]
    else:
        s = np.reciprocal(1.0 + np.exp(-x))
    a = s[rows, ids]
    if st["renorm"]:                                     # w_i = a_i / A
        A = a.sum(1)[:, None]
        g = g / A - ((g * a).sum(1)[:, None]) / (A * A)
    out = np.zeros_like(s)
    if st["score"] == "softmax":                         # ds_i / dx_e = s_i (1[i = e] - s_e)
        out -= s * (g * a).sum(1)[:, None]
        out[rows, ids] += g * a
    else:
        out[rows, ids] = g * a * (1.0 - a)
    return torch.from_numpy(out).cuda()


def _exact_dispatch(st):
    ids = st["ids"].cpu().numpy()
    T, k = ids.shape
    E, rows = st["E"], _rows(T, k, st["E"])
    by_expert = [[] for _ in range(E)]
    for p, e in enumerate(ids.reshape(-1).tolist()):
        by_expert[e].append(p)
    offsets, counts = np.zeros(E + 1, np.int32), np.zeros(E, np.int32)
    row_token, pair_row = np.full(rows, -1, np.int64), np.zeros(T * k, np.int32)
    for e, members in enumerate(by_expert):
        at, counts[e] = int(offsets[e]), len(members)
        offsets[e + 1] = at + -(-len(members) // PAD) * PAD
        members = np.array(members, np.int64)
        pair_row[members] = at + np.arange(len(members))
        row_token[at:at + len(members)] = members // k
    return tuple(torch.from_numpy(a).cuda() for a in (offsets, counts, row_token, pair_row.reshape(T, k)))


def _exact_combine(st):
    out = torch.zeros((st["T"], st["H"]), dtype=torch.float64, device="cuda")
    for j in range(st["k"]):
        out += st["weights"][:, j:j + 1].double() * st["y"][st["pair_row"][:, j].long()].double()
    return out


def _exact_combine_grad(st):
    d_y = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
    d_w = torch.zeros((st["T"], st["k"]), dtype=torch.float64, device="cuda")
    d = st["d_out"].double()
    for j in range(st["k"]):
        row = st["pair_row"][:, j].long()
        d_y[row] = st["weights"][:, j:j + 1].double() * d
        d_w[:, j] = (d * st["y"][row].double()).sum(1)
    return d_y, d_w


def _exact_logprobs(st):
    T, n = st["T"], st["top"]
    lp, H = (torch.zeros(T, dtype=torch.float64, device="cuda") for _ in range(2))
    stats = torch.zeros((T, 2), dtype=torch.float64, device="cuda")
    top, ids = torch.zeros((T, n), dtype=torch.float64, device="cuda"), None
    if n:
        ids = torch.zeros((T, n), dtype=torch.int64, device="cuda")
    step = max(1, (1 << 26) // st["V"])
    for a in range(0, T, step):
        b = min(T, a + step)
        z = st["logits"][a:b].double() / st["temperature"]
        m = torch.amax(z, 1)
        q = torch.exp(z - m[:, None])
        tot = q.sum(1)
        q = q / tot[:, None]
        logq = torch.log(torch.where(q > 0, q, 1.0))
        H[a:b] = -(q * logq).sum(1)
        stats[a:b, 0], stats[a:b, 1] = m, torch.log(tot)
        t = st["targets"][a:b]
        for_target = z[torch.arange(b - a, device="cuda"), t.clamp_min(0)]
        lp[a:b] = torch.where(t >= 0, for_target - m - torch.log(tot), 0.0)
        if n:
            left = st["logits"][a:b].double().clone()
            column = torch.arange(st["V"], device="cuda")[None]
            for i in range(n):                           # the lowest column that holds the largest value left
                first = torch.where(left == torch.amax(left, 1)[:, None], column, st["V"]).amin(1)
                ids[a:b, i] = first
                top[a:b, i] = z[torch.arange(b - a, device="cuda"), first] - m - torch.log(tot)
                left.scatter_(1, first[:, None], -math.inf)
    return (lp, H, stats, top, ids) if n else (lp, H, stats)


def _exact_logprobs_grad(st):
    out = torch.empty(st["logits"].shape, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // st["V"])
    for a in range(0, st["T"], step):
        b = min(st["T"], a + step)
        z = st["logits"][a:b].double() / st["temperature"]
        q = torch.softmax(z, 1)
        logq = torch.log(torch.where(q > 0, q, 1.0))
        H = -(q * logq).sum(1, keepdim=True)
        t = st["targets"][a:b, None]
        g = torch.where(t >= 0, st["d_logprobs"][a:b, None].double(), 0.0)
        d = -q * (g + st["d_entropy"][a:b, None].double() * (logq + H))
        d.scatter_add_(1, t.clamp_min(0), g)
        out[a:b] = d / st["temperature"]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(st)
    if op == "route_grad":
        return _exact_route_grad(st)
    if op == "dispatch":
        return _exact_dispatch(st)
    if op == "combine":
        return _exact_combine(st)
    if op == "combine_grad":
        return _exact_combine_grad(st)
    if op == "logprobs":
        return _exact_logprobs(st)
    return _exact_logprobs_grad(st)
