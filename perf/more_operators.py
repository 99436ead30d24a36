"""The measured cases of the 8-bit activation checkpoints, the low-rank
adapters and the verification of drafted tokens, with their plain forms.

``run`` computes an operator either in its plain form (elementary torch
operations in fp32, fp64 where a comparison decides) or, with ``own`` true,
through this package's calls.  ``exact`` gives the same outputs in fp64 from
the definitions.

Operators (``case["op"]``):
  swiglu         silu(gate) * up, with gate and up kept as MXFP8 for the backward pass
  swiglu_grad    its gradient from the 8-bit checkpoint, and the product again
  lora           rows of many requests through their own low-rank adapters, added to a shared projection's output
  lora_grad      the adapters' gradients and their share of the input's
  verify         drafted tokens accepted or refused, and the token that follows
"""
import math

import torch

own = False

BLOCK = 32               # elements that share an MXFP8 scale
PAD = 32                 # rows of an adapter's group are padded to this multiple

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_ESIZE = {"f32": 4, "bf16": 2}
GRID = 1 + 1 / BLOCK     # bytes of an element held as MXFP8


def listed():
    return [
        # a few rows of an expert: pure latency
        dict(name="swiglu_expert", op="swiglu", T=33, I=768, h="bf16"),
        # the MLP of a training micro-batch, its product quantized for the down projection
        dict(name="swiglu_mlp", op="swiglu", T=8192, I=12288, h="grid"),
        # the expert rows of a training micro-batch, backwards
        dict(name="swiglu_grad_experts", op="swiglu_grad", T=65568, I=768),
        # the MLP of an odd number of tokens, backwards
        dict(name="swiglu_grad_mlp", op="swiglu_grad", T=4095, I=12288),
        # one token of one request: pure latency
        dict(name="lora_token", op="lora", T=1, n=8, r=16, K=4096, N=6144, dtype="bf16", none=False),
        # a serving batch: many requests, many adapters, some requests without one
        dict(name="lora_serve", op="lora", T=250, n=64, r=16, K=4096, N=6144, dtype="bf16", none=True),
        # a training micro-batch of one adapter
        dict(name="lora_train", op="lora", T=8192, n=1, r=64, K=4096, N=6144, dtype="bf16", none=False),
        # the gradients of several adapters trained at once, inputs kept in bf16
        dict(name="lora_grad_mixed", op="lora_grad", T=4001, n=8, r=16, K=2048, N=1536, x="bf16"),
        # the gradients of one adapter, inputs kept as the MXFP8 operand of the shared projection
        dict(name="lora_grad_train", op="lora_grad", T=8192, n=1, r=32, K=4096, N=6144, x="grid"),
        # one request with four drafted tokens: latency
        dict(name="verify_one", op="verify", B=1, n=4, ragged=False, V=131072, dtype="bf16", draft=True, temperature=1.0),
        # a serving batch, up to seven drafted tokens a request, some with none
        dict(name="verify_batch", op="verify", B=64, n=7, ragged=True, V=131072, dtype="bf16", draft=True,
             temperature=0.7),
        # tokens looked up in the prompt (no draft distribution), fp32 logits, odd vocabulary
        dict(name="verify_lookup", op="verify", B=33, n=5, ragged=False, V=100003, dtype="f32", draft=False,
             temperature=1.0),
    ]


def _log_int(rng, lo, hi):
    # spread over the logarithm; whole multiples of 1024 are left to the listed cases
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n if n % 1024 else n - 1


def draw(rng):
    op = rng.choice(["swiglu", "swiglu_grad", "lora", "lora_grad", "verify"])
    if op in ("swiglu", "swiglu_grad"):
        inner = BLOCK * _log_int(rng, 1, 384)
        T = _log_int(rng, 1, min(65536, 8192 * 12288 // inner))
        case = dict(op=op, T=T, I=inner)
        if op == "swiglu":
            case["h"] = rng.choice(["bf16", "grid"])
        return case
    if op in ("lora", "lora_grad"):
        r = 8 * rng.choice([1, 1, 2, 2, 3, 4, 6, 8])
        n = rng.choice([1, 1, _log_int(rng, 2, 512 // r)])
        K, N = BLOCK * _log_int(rng, 2, 128), 8 * _log_int(rng, 8, 768)
        T = _log_int(rng, 1, max(2, min(8192, 8192 * 64 * 10240 // (n * r * (K + N)))))
        case = dict(op=op, T=T, n=n, r=r, K=K, N=N)
        if op == "lora":
            return dict(case, dtype=rng.choice(["bf16", "bf16", "f32"]), none=rng.random() < 0.4)
        return dict(case, x=rng.choice(["bf16", "grid"]))
    V, n = _log_int(rng, 1000, 131072), rng.randint(1, 7)
    B = _log_int(rng, 1, min(64, max(2, 64 * 131072 // V)))
    return dict(op=op, B=B, n=n, ragged=rng.random() < 0.5, V=V, dtype=rng.choice(["f32", "bf16"]),
                draft=rng.random() < 0.6, temperature=rng.choice([1.0, 0.7, 1.3]))


def _drafts(case):
    """Drafted tokens of each request."""
    n = case["n"]
    return [(5 * b + 3) % (n + 1) if case["ragged"] else n for b in range(case["B"])]


def _group_rows(T, n):
    """Rows that the padded groups of T rows over n adapters can take at most."""
    return (T + min(n, T) * (PAD - 1)) // PAD * PAD


def work(case):
    op = case["op"]
    if op == "swiglu":
        n = case["T"] * case["I"]
        return {"bytes": n * (4 + 2 * GRID + (2 if case["h"] == "bf16" else GRID)), "flops": 10 * n}
    if op == "swiglu_grad":
        n = case["T"] * case["I"]
        return {"bytes": n * (2 + 2 * GRID + 4 + 2), "flops": 15 * n}
    if op in ("lora", "lora_grad"):
        T, n, r, K, N = (case[k] for k in ("T", "n", "r", "K", "N"))
        weights = min(n, T) * r * (K + N) * 2
        if op == "lora":
            return {"bytes": T * K * 2 + 2 * T * N * _ESIZE[case["dtype"]] + weights + T * r * 4,
                    "flops": 2 * T * r * (K + N)}
        x = T * K * (2 if case["x"] == "bf16" else GRID)
        return {"bytes": x + T * N * 2 + 2 * T * K * 2 + T * r * 4 + weights + n * r * (K + N) * 4,
                "flops": 4 * T * r * (K + N)}
    B, V, D = case["B"], case["V"], sum(_drafts(case))
    rows = B + D + (D if case["draft"] else 0)
    return {"bytes": rows * V * _ESIZE[case["dtype"]] + B * V * 4 + D * 12, "flops": 4 * rows * V + 8 * B * V}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(shape, g, factor):
    # now and then a value far larger than its neighbours
    x = torch.randn(shape, generator=g, device="cuda")
    return torch.where(torch.rand(shape, generator=g, device="cuda") < 0.01, x * factor, x).to(torch.bfloat16)


def _tables(ids, n):
    """The rows of every adapter together, each adapter's padded: offsets [n + 1], row_token [rows]."""
    T, rows = ids.numel(), _group_rows(ids.numel(), n)
    real = (ids >= 0) & (ids < n)
    key = torch.where(real, ids.long(), n)
    counts = torch.zeros(n + 1, dtype=torch.long, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    padded = (counts + PAD - 1) // PAD * PAD
    start = torch.cumsum(padded, 0) - padded
    order = torch.sort(key, stable=True).indices
    expert = key[order]
    place = start[expert] + torch.arange(T, device=ids.device) - (torch.cumsum(counts, 0) - counts)[expert]
    row_token = torch.full((rows + T + PAD,), -1, dtype=torch.long, device=ids.device)
    row_token[torch.where(expert < n, place, rows + torch.arange(T, device=ids.device))] = order
    row_token[rows:] = -1
    return start.to(torch.int32), counts[:n].to(torch.int32), row_token[:rows].contiguous()


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    st = dict(case)
    if op in ("swiglu", "swiglu_grad"):
        T, inner = case["T"], case["I"]
        gu = _activations((T, 2 * inner), g, 6.0)
        if op == "swiglu":
            st["gu"] = gu
            return st
        st["q"], st["s"] = _plain_quantize(gu)
        st["d_h"] = (torch.randn((T, inner), generator=g, device="cuda") * 2.0 ** -8).to(torch.bfloat16)
        return st
    if op in ("lora", "lora_grad"):
        T, n, r, K, N = (case[k] for k in ("T", "n", "r", "K", "N"))
        # requests hold runs of rows; adapters differ in popularity
        run = max(1, T // 64)
        pick = (torch.rand((T + run - 1) // run, generator=g, device="cuda") ** 1.6 * n).long().clamp_max(n - 1)
        if case.get("none"):
            pick = torch.where(torch.rand(pick.numel(), generator=g, device="cuda") < 0.2, -1, pick)
        ids = pick.repeat_interleave(run)[:T].to(torch.int32)
        st["ids"] = ids
        st["offsets"], st["counts"], st["row_token"] = _tables(ids, n)
        x = _activations((T, K), g, 20.0)
        st["a"] = (torch.randn((n, r, K), generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16)
        st["b"] = (torch.randn((n, N, r), generator=g, device="cuda") * 0.02).to(torch.bfloat16)
        st["scales"] = 0.5 + torch.rand(n, generator=g, device="cuda")
        if op == "lora":
            st["x"] = x
            st["y"] = torch.randn((T, N), generator=g, device="cuda").to(_TYPES[case["dtype"]])
            return st
        if case["x"] == "grid":
            st["xq"], st["xs"] = _plain_quantize(x)
            x = _plain_values(st["xq"], st["xs"]).to(torch.bfloat16)
        st["input"] = x
        if case["x"] == "bf16":
            st["x_bf16"] = x
        st["hidden"] = _rows_of(_plain_hidden(st["input"], st["a"], ids).sum(1), st["row_token"])
        del st["input"]
        st["d_y"] = (torch.randn((T, N), generator=g, device="cuda") * 2.0 ** -8).to(torch.bfloat16)
        st["d_x"] = (torch.randn((T, K), generator=g, device="cuda") * 2.0 ** -8).to(torch.bfloat16)
        return st
    B, V, t = case["B"], case["V"], _TYPES[case["dtype"]]
    counts = _drafts(case)
    D = sum(counts)
    R = B + D
    st["offsets"] = torch.tensor([0] + [sum(counts[:b + 1]) + b + 1 for b in range(B)], dtype=torch.int32, device="cuda")
    # a few likely continuations stand out at every position
    x = torch.randn((R, V), generator=g, device="cuda") * 2.0
    used = V - V // 1024
    part = used // 24
    likely = torch.randint(0, part, (R, 24), generator=g, device="cuda") + part * torch.arange(24, device="cuda")
    x.scatter_(1, likely, 4.0 + 9.0 * torch.rand((R, 24), generator=g, device="cuda"))
    x[:, used:] = -math.inf                              # ids that the tokenizer does not use
    st["logits"] = x.to(t)
    drafted = torch.ones(R, dtype=torch.bool, device="cuda")
    drafted[st["offsets"][1:].long() - 1] = False
    # the draft model agrees with the target up to some noise, and draws its tokens from its own distribution
    z = x[drafted]
    z = (z + torch.randn(z.shape, generator=g, device="cuda") * 0.7).to(t)
    race = torch.empty((D, V), device="cuda").exponential_(generator=g)
    st["draft_ids"] = torch.argmax(z.float() / case["temperature"] - torch.log(race), 1) if D else torch.zeros(
        0, dtype=torch.long, device="cuda")
    st["draft_logits"] = z if case["draft"] else None
    st["uniforms"] = torch.rand(D, generator=g, device="cuda")
    st["noise"] = torch.empty((B, V), device="cuda").exponential_(generator=g).clamp_min_(2.0 ** -24)
    return st


# ------------------------------------------------------------------ plain forms

def _power(e):
    """2^e in fp32, exact, for whole e of -126 to 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _plain_quantize(x):
    """bf16 [T, C] -> E4M3 codes and one power-of-two scale code per 32 values of a row."""
    T, C = x.shape
    v = x.float().view(T, C // BLOCK, BLOCK)
    amax = v.abs().amax(2)
    exponent = torch.where(amax > 0, torch.frexp(amax).exponent - 9, -127).clamp_min(-127)      # floor(log2 amax) - 8
    v = (v * _power(-exponent.unsqueeze(2))).clamp(-448.0, 448.0)
    step = _power(torch.frexp(v).exponent.clamp_min(-5) - 4)
    v = torch.round(v / step) * step
    return v.view(T, C).to(torch.float8_e4m3fn).view(torch.uint8), (exponent + 127).to(torch.uint8)


def _plain_values(q, s):
    T, C = q.shape
    v = q.view(torch.float8_e4m3fn).float().view(T, C // BLOCK, BLOCK)
    e = s.int().unsqueeze(2) - 127
    return (v * _power(e.clamp_min(-126)) * torch.where(e < -126, 0.5, 1.0)).view(T, C)


def _as_values(q, s):
    """Codes and scales as the numbers they stand for."""
    return q.view(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu)


def _plain_swiglu(st):
    q, s = _plain_quantize(st["gu"])
    g, u = st["gu"].float().chunk(2, 1)
    h = (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)
    saved = _as_values(q, s)
    return saved + (h,) if st["h"] == "bf16" else saved + _as_values(*_plain_quantize(h))


def _plain_swiglu_grad(st):
    g, u = _plain_values(st["q"], st["s"]).chunk(2, 1)
    d = st["d_h"].float()
    sig = 1 / (1 + torch.exp(-g))
    d_gu = torch.cat((d * u * sig * (1 + g * (1 - sig)), d * g * sig), 1)
    return d_gu.to(torch.bfloat16), (g * sig * u).to(torch.bfloat16)


def _plain_hidden(x, a, ids):
    """A x of every row and adapter, zeros but for the row's own: [T, n, r]."""
    n, r, K = a.shape
    h = (x.float() @ a.float().view(n * r, K).t()).view(-1, n, r)
    return torch.where((ids.unsqueeze(1) == torch.arange(n, device=ids.device)).unsqueeze(2), h, 0.0)


def _rows_of(h, row_token):
    return torch.where(row_token.unsqueeze(1) >= 0, h[row_token.clamp_min(0)], 0.0)


def _plain_lora(st):
    a, b, ids, y = st["a"], st["b"], st["ids"], st["y"]
    n, N, r = b.shape
    h = _plain_hidden(st["x"], a, ids)
    scaled = (h * st["scales"].view(1, n, 1)).reshape(-1, n * r)
    y.copy_(y.float() + scaled @ b.float().permute(0, 2, 1).reshape(n * r, N))
    return y, _rows_of(h.sum(1), st["row_token"])


def _plain_lora_grad(st):
    a, b, ids, d_y = st["a"].float(), st["b"].float(), st["ids"], st["d_y"].float()
    n, r, K = a.shape
    N, T = b.shape[1], ids.numel()
    x = st["x_bf16"].float() if st["x"] == "bf16" else _plain_values(st["xq"], st["xs"])
    mine = (ids.unsqueeze(1) == torch.arange(n, device=ids.device)).unsqueeze(2)
    weight = torch.where(mine, st["scales"].view(1, n, 1), 0.0)
    s = ((d_y @ b.permute(1, 0, 2).reshape(N, n * r)).view(T, n, r) * weight).view(T, n * r)
    st["d_x"].copy_(st["d_x"].float() + s @ a.view(n * r, K))
    d_a = (s.t() @ x).view(n, r, K)
    row = st["row_token"]
    h = torch.zeros((T, r), device=row.device).index_add_(0, row.clamp_min(0), st["hidden"])
    d_b = (d_y.t() @ (h.unsqueeze(1) * weight).view(T, n * r)).view(N, n, r).permute(1, 0, 2).contiguous()
    return st["d_x"], d_a, d_b


def _plain_softmax64(x, temperature):
    z = x.double() / temperature
    z = z - z.amax(1, keepdim=True)
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    return e / total, z - torch.log(total)


def _plain_verify(st):
    # the decisions in fp64: values that differ below fp32's step still have an order
    off, ids, V = st["offsets"].long(), st["draft_ids"], st["V"]
    B, D = off.numel() - 1, ids.numel()
    R = B + D
    p, logp = _plain_softmax64(st["logits"], st["temperature"])
    row = torch.arange(R, device=off.device)
    request = torch.searchsorted(off[1:].contiguous(), row, right=True)
    position = row - off[request]
    last = off[1:] - 1
    drafted = row != last[request]
    at = row[drafted]
    px = p[at, ids]
    if st["draft_logits"] is None:
        q, qx = None, torch.ones_like(px)
    else:
        q, _ = _plain_softmax64(st["draft_logits"], st["temperature"])
        qx = q.gather(1, ids.unsqueeze(1)).squeeze(1)
    refused = ~(st["uniforms"].double() * qx < px)
    end = (last - off[:-1]).clone()
    end.scatter_reduce_(0, request[at], torch.where(refused, position[at], V), "amin")
    chosen = off[:-1] + end
    stopped = chosen < last
    rest = p[chosen]
    if D:
        slot = (chosen - torch.arange(B, device=off.device)).clamp(0, D - 1)
        if q is None:
            taken = torch.zeros_like(rest).scatter_(1, ids[slot].unsqueeze(1), 1.0)
        else:
            taken = q[slot]
        rest = torch.where(stopped.unsqueeze(1), rest - taken, rest)
    score = torch.where(rest > 0, rest / st["noise"].double(), 0.0)
    column = torch.arange(V, device=off.device)
    token = torch.where(score == score.amax(1, keepdim=True), column, V).amin(1)
    tokens = torch.full((R,), -1, dtype=torch.long, device=off.device)
    tokens[at] = torch.where(position[at] < end[request[at]], ids, -1)
    tokens[chosen] = token
    logprobs = torch.where(tokens >= 0, logp.gather(1, tokens.clamp_min(0).unsqueeze(1)).squeeze(1), 0.0)
    return end.to(torch.int32), tokens, logprobs.float()


# ------------------------------------------------------------------ one pass

def _run_own(st):
    import mxfp8_block_scaled_05_amd as mx
    op = st["op"]
    if op == "swiglu":
        if st["h"] == "bf16":
            r = mx.swiglu(st["gu"])
            return _as_values(r.saved_q, r.saved_s) + (r.h,)
        r = mx.swiglu(st["gu"], layout="canonical")
        return _as_values(r.saved_q, r.saved_s) + _as_values(*r.h)
    if op == "swiglu_grad":
        return mx.swiglu_backward(st["d_h"], st["q"], st["s"])
    if op in ("lora", "lora_grad"):
        tables = mx.RouteTables(st["offsets"], st["counts"], st["row_token"], None, PAD)
        if op == "lora":
            hidden = mx.lora_add_(st["y"], st["x"], st["a"], st["b"], tables, st["scales"], keep_hidden=True)
            return st["y"], hidden
        x = st["x_bf16"] if st["x"] == "bf16" else (st["xq"], st["xs"])
        d_a, d_b = mx.lora_backward_(st["d_x"], st["d_y"], x, st["a"], st["b"], st["hidden"], tables, st["scales"])
        return st["d_x"], d_a, d_b
    r = mx.verify_drafts(st["logits"], st["offsets"], st["draft_ids"], st["uniforms"], st["noise"],
                         draft_logits=st["draft_logits"], temperature=st["temperature"])
    return r.accepted, r.tokens, r.logprobs


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "swiglu":
        return _plain_swiglu(state)
    if op == "swiglu_grad":
        return _plain_swiglu_grad(state)
    if op == "lora":
        return _plain_lora(state)
    if op == "lora_grad":
        return _plain_lora_grad(state)
    return _plain_verify(state)


# ------------------------------------------------------------------ fp64 definitions

def _magnitudes():
    """The 127 finite magnitudes of E4M3, by rising code."""
    at = [(c % 8 + (8 if c >= 8 else 0), max(c // 8, 1) - 10) for c in range(127)]
    return torch.tensor([math.ldexp(m, e) for m, e in at], dtype=torch.float64, device="cuda")


def _powers():
    """2^-127 to 2^127 (a power function rounds)."""
    return torch.tensor([math.ldexp(1.0, k) for k in range(-127, 128)], dtype=torch.float64, device="cuda")


def _exact_grid(x):
    """The values of an MXFP8 grid of x: nearest E4M3 magnitude, the even code between two."""
    table, powers = _magnitudes(), _powers()
    middle = (table[1:] + table[:-1]) / 2
    q = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    scale = torch.empty((x.shape[0], x.shape[1] // BLOCK), dtype=torch.float64, device="cuda")
    rows = max(1, (1 << 24) // x.shape[1])
    for i in range(0, x.shape[0], rows):
        v = x[i:i + rows].double().view(-1, x.shape[1] // BLOCK, BLOCK)
        amax = torch.amax(torch.abs(v), 2, keepdim=True)
        # the entry of the largest power up to amax, and the one 8 below it
        power = torch.searchsorted(powers, amax, right=True) - 1 - 8
        power = power.clamp_min(0)
        v = v / powers[power]
        size = torch.abs(v)
        low = torch.searchsorted(middle, size)
        tie = (low < 126) & (middle[low.clamp_max(125)] == size) & (low % 2 == 1)
        q[i:i + rows] = (torch.sign(v) * table[torch.where(tie, low + 1, low)]).reshape(-1, x.shape[1])
        scale[i:i + rows] = powers[power].squeeze(2)
    return q, scale


def _exact_swiglu(st):
    gu, inner = st["gu"], st["I"]
    h = torch.nn.functional.silu(gu[:, :inner].double()) * gu[:, inner:].double()
    if st["h"] == "bf16":
        return _exact_grid(gu) + (h,)
    return _exact_grid(gu) + _exact_grid(h.to(torch.bfloat16))


def _exact_swiglu_grad(st):
    T, inner = st["T"], st["I"]
    d_gu = torch.empty((T, 2 * inner), dtype=torch.float64, device="cuda")
    h = torch.empty((T, inner), dtype=torch.float64, device="cuda")
    scale = _powers()[st["s"].long()]
    rows = max(1, (1 << 24) // inner)
    for i in range(0, T, rows):
        v = st["q"][i:i + rows].view(torch.float8_e4m3fn).double() * scale[i:i + rows].repeat_interleave(BLOCK, 1)
        g, u, d = v[:, :inner], v[:, inner:], st["d_h"][i:i + rows].double()
        e = torch.sigmoid(g)
        h[i:i + rows] = g * e * u
        d_gu[i:i + rows, :inner] = d * u * (e + g * e * torch.sigmoid(-g))      # (g e)' = e + g e (1 - e)
        d_gu[i:i + rows, inner:] = d * g * e
    return d_gu, h


def _exact_rows(st):
    """(adapter, its rows) for the adapters that have any."""
    return [(e, torch.nonzero(st["ids"] == e).squeeze(1)) for e in torch.unique(st["ids"]).tolist() if e >= 0]


def _exact_lora(st):
    y = st["y"].double()
    h = torch.zeros((st["T"], st["r"]), dtype=torch.float64, device="cuda")
    for e, t in _exact_rows(st):
        h[t] = torch.nn.functional.linear(st["x"][t].double(), st["a"][e].double())
        y[t] += st["scales"][e].double() * torch.nn.functional.linear(h[t], st["b"][e].double())
    out = torch.zeros((st["row_token"].numel(), st["r"]), dtype=torch.float64, device="cuda")
    held = st["row_token"] >= 0
    out[held] = h[st["row_token"][held]]
    return y, out


def _exact_lora_grad(st):
    if st["x"] == "bf16":
        x = st["x_bf16"].double()
    else:
        x = st["xq"].view(torch.float8_e4m3fn).double() * _powers()[st["xs"].long()].repeat_interleave(BLOCK, 1)
    d_x = st["d_x"].double()
    d_a = torch.zeros(st["a"].shape, dtype=torch.float64, device="cuda")
    d_b = torch.zeros(st["b"].shape, dtype=torch.float64, device="cuda")
    held = st["row_token"] >= 0
    h = torch.zeros((st["T"], st["r"]), dtype=torch.float64, device="cuda")
    h[st["row_token"][held]] = st["hidden"][held].double()
    for e, t in _exact_rows(st):
        a, b, dy = st["a"][e].double(), st["b"][e].double(), st["d_y"][t].double() * st["scales"][e].double()
        dh = torch.matmul(dy, b)
        d_x[t] += torch.matmul(dh, a)
        d_a[e] = torch.matmul(dh.t().contiguous(), x[t])
        d_b[e] = torch.matmul(dy.t().contiguous(), h[t])
    return d_x, d_a, d_b


def _exact_verify(st):
    off, ids, u = st["offsets"].tolist(), st["draft_ids"].tolist(), st["uniforms"].tolist()
    accepted, tokens, logprobs = [], [-1] * st["logits"].shape[0], [0.0] * st["logits"].shape[0]

    def log_softmax(x):
        return torch.log_softmax(x.double() / st["temperature"], 0)

    for b in range(st["B"]):
        drafts, count = off[b + 1] - off[b] - 1, 0
        while True:
            i, slot = off[b] + count, off[b] - b + count
            lp = log_softmax(st["logits"][i])
            rest = torch.exp(lp)
            if count == drafts:
                break
            x = ids[slot]
            q = torch.zeros_like(rest)
            if st["draft_logits"] is None:
                q[x] = 1.0
            else:
                q = torch.exp(log_softmax(st["draft_logits"][slot]))
            if u[slot] * q[x].item() >= rest[x].item():
                rest = torch.clamp_min(rest - q, 0.0)
                break
            tokens[i], logprobs[i] = x, lp[x].item()
            count += 1
        score = rest / st["noise"][b].double()
        token = int(torch.nonzero(score == score.max())[0])
        tokens[i], logprobs[i] = token, lp[token].item()
        accepted.append(count)
    return (torch.tensor(accepted, dtype=torch.int32, device="cuda"), torch.tensor(tokens, device="cuda"),
            torch.tensor(logprobs, dtype=torch.float64, device="cuda"))


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "swiglu":
        return _exact_swiglu(st)
    if op == "swiglu_grad":
        return _exact_swiglu_grad(st)
    if op == "lora":
        return _exact_lora(st)
    if op == "lora_grad":
        return _exact_lora_grad(st)
    return _exact_verify(st)
