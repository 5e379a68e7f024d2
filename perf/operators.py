"""The operators of a linear-attention layer as it is served, in plain torch and as this library's calls.

  rms_norm               x + residual, root-mean-square norm, output in bf16, fp32, or e4m3 with a scale for
                         each 128 columns of a row
  matmul_fp8             e4m3 times e4m3 with a scale for each 128 columns of a row of the activations and
                         each 128 x 128 block of the weights
  linear_attention       causal linear attention with a decay for each head over whole prompts (chunked)
  linear_attention_step  the same recurrence for one new token of each sequence, on a pool of states

`run` computes them in plain torch where `own` is false, and calls selective_scan_02_b200 where it is true.
"""
import math

import torch

own = False

EPS = 1e-6
BLOCK = 128
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100


def listed():
    return [
        # the norm before a decode step's projections: a few rows, where latency counts
        dict(name="norm_decode", op="norm", rows=8, dim=4096, x="bf16", residual="f32", out="e4m3"),
        # the same norm over a long prompt, residual stream in bf16
        dict(name="norm_prompt", op="norm", rows=16384, dim=4096, x="bf16", residual="bf16", out="e4m3"),
        # between two SS2D blocks of the stage-1 workload (batch 32, 56 x 56 pixels, d_model 96), all fp32, bf16 out
        dict(name="norm_image", op="norm", rows=32 * 56 * 56, dim=96, x="f32", residual="f32", out="bf16"),
        # the fused q, k, v projection of four sequences' new tokens: the weights' bytes are the work
        dict(name="matmul_decode", op="matmul", m=4, n=6144, k=2048, bias=False, out="bf16"),
        # a ragged batch of short prompts, fp32 out: no size is a multiple of a tile
        dict(name="matmul_ragged", op="matmul", m=333, n=1000, k=1104, bias=True, out="f32"),
        # a long prompt through a wide projection
        dict(name="matmul_prompt", op="matmul", m=8192, n=6144, k=4096, bias=False, out="bf16"),
        # one long prompt with few heads and a fixed decay for each
        dict(name="attention_long", op="attention", b=1, l=32768, g=16, h=16, dk=128, dv=128, gates="head",
             ragged=False, h0=False, fused=False),
        # image tokens in scan order (batch 32, 56 x 56 pixels, 192 channels as 6 heads of 32), q and k shared by the
        # heads and a decay for each token
        dict(name="attention_image", op="attention", b=32, l=56 * 56, g=1, h=6, dk=64, dv=32, gates="token",
             ragged=False, h0=False, fused=True),
        # prompts of different lengths, each continued from a state: padded rows behind each
        dict(name="attention_ragged", op="attention", b=7, l=1531, g=8, h=32, dk=128, dv=64, gates="token",
             ragged=True, h0=True, fused=True),
        # one sequence's new token
        dict(name="step_one", op="step", b=1, pool=1, g=16, h=16, dk=128, dv=128, gates="head", slots=False,
             fused=False),
        # a full batch's new tokens
        dict(name="step_batch", op="step", b=64, pool=64, g=32, h=32, dk=128, dv=128, gates="head", slots=False,
             fused=True),
        # new tokens of the sequences in hand: states picked from a pool, some rows of the batch empty
        dict(name="step_pool", op="step", b=33, pool=48, g=8, h=24, dk=64, dv=96, gates="token", slots=True,
             fused=True),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "matmul", "attention", "step"])
    if op == "norm":
        dim = rng.choice([_spread(rng, 1, 256), 8 * _spread(rng, 4, 1024)])
        rows = _spread(rng, 1, max(1, min(100352, 2 ** 26 // dim)))
        return dict(op=op, rows=rows, dim=dim, x=rng.choice(["bf16", "f32"]),
                    residual=rng.choice(["none", "bf16", "f32"]), out=rng.choice(["bf16", "f32", "e4m3"]))
    if op == "matmul":
        m, n, k = _spread(rng, 1, 8192), _spread(rng, 8, 8192), 16 * _spread(rng, 1, 512)
        while m * n * k > 2 ** 37:
            m = (m + 1) // 2
        return dict(op=op, m=m, n=n, k=k, bias=rng.random() < 0.3,
                    out=rng.choice(["bf16", "bf16", "f32"]))
    h = _spread(rng, 1, 32)
    g = rng.choice([d for d in range(1, h + 1) if h % d == 0])
    dk, dv = 8 * _spread(rng, 2, 16), 8 * _spread(rng, 2, 16)
    case = dict(op=op, g=g, h=h, dk=dk, dv=dv, gates=rng.choice(["head", "token"]), fused=rng.random() < 0.5)
    if op == "attention":
        b = _spread(rng, 1, 16)
        top = max(2, min(32768, 2 ** 26 // (b * (g * dk + h * dv) * 2)))
        return dict(case, b=b, l=_spread(rng, 1, top), ragged=rng.random() < 0.4, h0=rng.random() < 0.5)
    b = _spread(rng, 1, 128)
    while b * h * dk * dv > 2 ** 25:
        b = (b + 1) // 2
    slots = rng.random() < 0.5
    return dict(case, b=b, pool=b + rng.randrange(0, 16) if slots else b, slots=slots)


TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def _decays(case, shape, gen):
    """log_decay: fixed for each head (slow heads remember thousands of tokens, fast ones tens), or one for each
    token and head, from a softplus of what a projection gives times a rate of each head."""
    h = case["h"]
    steps = torch.arange(h, device="cuda", dtype=torch.float32)
    if case["gates"] == "head":
        return torch.log1p(-torch.exp2(-3.0 - 8.0 * (steps + torch.rand(h, device="cuda", generator=gen)) / h))
    rate = torch.exp(torch.rand(h, device="cuda", generator=gen) * 2.7)
    x = torch.randn(shape, device="cuda", generator=gen) - 3.0
    return -rate * torch.nn.functional.softplus(x)


def _qkv(case, lead, gen):
    """q, k (lead, g, dk) and v (lead, h, dv): columns of one projection's output, or three tensors."""
    g, h, dk, dv = case["g"], case["h"], case["dk"], case["dv"]
    widths = [g * dk, g * dk, h * dv]
    if case["fused"]:
        parts = torch.randn(*lead, sum(widths), device="cuda", generator=gen).bfloat16().split(widths, dim=-1)
    else:
        parts = [torch.randn(*lead, w, device="cuda", generator=gen).bfloat16() for w in widths]
    q, k, v = (p.unflatten(-1, s) for p, s in zip(parts, [(g, dk), (g, dk), (h, dv)]))
    return q, k, v


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "norm":
        r, d = case["rows"], case["dim"]
        x = torch.randn(r, d, device="cuda", generator=gen).to(TYPES[case["x"]])
        weight = 1.0 + 0.2 * torch.randn(d, device="cuda", generator=gen)
        residual = None
        if case["residual"] != "none":
            residual = (3.0 * torch.randn(r, d, device="cuda", generator=gen)).to(TYPES[case["residual"]])
        return dict(op="norm", x=x, weight=weight, residual=residual, out=TYPES[case["out"]])
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        kb, nb = -(-k // BLOCK), -(-n // BLOCK)
        a = (90.0 * torch.randn(m, k, device="cuda", generator=gen)).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        w = (90.0 * torch.randn(n, k, device="cuda", generator=gen)).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        a_scales = torch.exp(0.5 * torch.randn(m, kb, device="cuda", generator=gen)) / 90.0
        w_scales = torch.exp(0.5 * torch.randn(nb, kb, device="cuda", generator=gen)) / (90.0 * math.sqrt(k))
        bias = torch.randn(n, device="cuda", generator=gen) if case["bias"] else None
        return dict(op="matmul", a=a, a_scales=a_scales, w=w, w_scales=w_scales, bias=bias, out=TYPES[case["out"]])
    b, h, dk, dv = case["b"], case["h"], case["dk"], case["dv"]
    if case["op"] == "attention":
        q, k, v = _qkv(case, (b, case["l"]), gen)
        log_decay = _decays(case, (b, case["l"], h), gen)
        h0 = torch.randn(b, h, dk, dv, device="cuda", generator=gen) if case["h0"] else None
        lengths = None
        if case["ragged"]:
            lengths = torch.randint(0, case["l"] + 1, (b,), device="cuda", generator=gen, dtype=torch.int32)
            lengths[0] = case["l"]
        out = torch.zeros(b, case["l"], h, dv, device="cuda", dtype=torch.bfloat16)
        return dict(op="attention", q=q, k=k, v=v, log_decay=log_decay, scale=dk ** -0.5, h0=h0, lengths=lengths,
                    out=out)
    q, k, v = _qkv(case, (b,), gen)
    log_decay = _decays(case, (b, h), gen)
    state = torch.randn(case["pool"], h, dk, dv, device="cuda", generator=gen)
    slots = None
    if case["slots"]:
        slots = torch.randperm(case["pool"], device="cuda", generator=gen)[:b].to(torch.int32)
        slots[torch.rand(b, device="cuda", generator=gen) < 0.1] = -1
    out = torch.zeros(b, h, dv, device="cuda", dtype=torch.bfloat16)
    return dict(op="step", q=q, k=k, v=v, log_decay=log_decay, scale=dk ** -0.5, state=state, slots=slots, out=out)


def run(s):
    if own:
        return _own(s)
    return {"norm": _norm, "matmul": _matmul, "attention": _attention, "step": _step}[s["op"]](s)


def _own(s):
    import selective_scan_02_b200 as ss

    if s["op"] == "norm":
        return ss.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, out_dtype=s["out"])
    if s["op"] == "matmul":
        return ss.matmul_fp8(s["a"], s["a_scales"], s["w"], s["w_scales"], bias=s["bias"], out_dtype=s["out"])
    if s["op"] == "attention":
        return ss.linear_attention(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"], h0=s["h0"],
                                   lengths=s["lengths"], return_last_state=True, out=s["out"])
    out = ss.linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], slots=s["slots"],
                                   scale=s["scale"], out=s["out"])
    return out, s["state"]


def _norm(s):
    r = s["x"].float()
    if s["residual"] is not None:
        r = r + s["residual"].float()
    y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * s["weight"]
    if s["out"] == torch.float8_e4m3fn:
        rows, d = y.shape
        kb = -(-d // BLOCK)
        blocks = torch.nn.functional.pad(y, (0, kb * BLOCK - d)).view(rows, kb, BLOCK)
        scales = (blocks.abs().amax(-1) / E4M3_MAX).clamp_min(SCALE_MIN)
        got = ((blocks / scales[..., None]).view(rows, -1)[:, :d].to(torch.float8_e4m3fn), scales)
    else:
        got = (y.to(s["out"]),)
    if s["residual"] is not None:
        got += (r.to(s["residual"].dtype),)
    return got if len(got) > 1 else got[0]


def _matmul(s):
    n, k = s["w"].shape
    a = s["a"].float() * s["a_scales"].repeat_interleave(BLOCK, dim=1)[:, :k]
    w = s["w"].float() * s["w_scales"].repeat_interleave(BLOCK, dim=0)[:n].repeat_interleave(BLOCK, dim=1)[:, :k]
    c = a @ w.t()
    if s["bias"] is not None:
        c = c + s["bias"]
    return c.to(s["out"])


def _attention(s):
    """Chunks of 128: within a chunk by the masked products, between chunks by the states at their ends."""
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    b, l, g, dk = q.shape
    h, dv = v.shape[2:]
    c = 128
    n = -(-l // c)
    gates = s["log_decay"].double()
    gates = gates.expand(b, l, h)
    real = torch.ones(b, l, dtype=torch.bool, device=q.device)
    if s["lengths"] is not None:
        real = torch.arange(l, device=q.device) < s["lengths"][:, None]
    gates = torch.where(real[..., None], gates, 0.0)
    k = torch.where(real[..., None, None], k, 0.0)
    v = torch.where(real[..., None, None], v, 0.0)

    def chunks(x):
        x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, n * c - l))
        return x.unflatten(1, (n, c)).movedim(3, 1)  # (b, heads, n, c, ...)

    q, k, v, gates = chunks(q), chunks(k), chunks(v), chunks(gates)
    cum = gates.cumsum(-1)                                   # decay from the chunk's start, (b, h, n, c)
    total = cum[..., -1]
    ends = total.cumsum(-1)                                  # from the first chunk's start, (b, h, n)
    tri = torch.ones(c, c, dtype=torch.bool, device=q.device).tril()
    weight = torch.where(tri, cum[..., :, None] - cum[..., None, :], -math.inf).exp().float()
    shared = lambda x: x.repeat_interleave(h // g, dim=1)  # noqa: E731
    scores = shared(q @ k.transpose(-1, -2)) * weight
    out = scores @ v
    del scores, weight
    local = shared(k).transpose(-1, -2) @ (v * (total[..., None] - cum).exp().float()[..., None])
    # state before chunk i: the chunks j < i, each decayed by what lies between its end and the start of i
    before = torch.ones(n, n, dtype=torch.bool, device=q.device).tril(-1)
    starts = ends - total
    carry = torch.where(before, starts[..., :, None] - ends[..., None, :], -math.inf).exp().float()
    states = (carry @ local.flatten(-2)).unflatten(-1, (dk, dv))
    last = ((ends[..., -1:] - ends).exp().float()[..., None, :] @ local.flatten(-2)).view(b, h, dk, dv)
    if s["h0"] is not None:
        states = states + starts.exp().float()[..., None, None] * s["h0"][:, :, None]
        last = last + ends[..., -1].exp().float()[..., None, None] * s["h0"]
    out = out + (shared(q) @ states) * cum.exp().float()[..., None]
    out = (out * s["scale"]).movedim(1, 3).flatten(1, 2)[:, :l].to(torch.bfloat16)
    s["out"].copy_(torch.where(real[..., None, None], out, s["out"]))
    return s["out"], last


def _step(s):
    q, k, v, state = s["q"].float(), s["k"].float(), s["v"].float(), s["state"]
    b, g, dk = q.shape
    h, dv = v.shape[1:]
    q, k = (x.repeat_interleave(h // g, dim=1) for x in (q, k))
    decay = s["log_decay"].expand(b, h).exp()[..., None, None]
    if s["slots"] is None:
        state.copy_(state * decay + k[..., None] * v[..., None, :])
        s["out"].copy_(((q[..., None] * state).sum(-2) * s["scale"]))
        return s["out"], state
    # rows without a slot are computed on a spare state, and what they give is left out
    spare = torch.cat([state, torch.zeros_like(state[:1])])
    at = torch.where(s["slots"] >= 0, s["slots"].long(), state.shape[0])
    new = spare[at] * decay + k[..., None] * v[..., None, :]
    out = ((q[..., None] * new).sum(-2) * s["scale"]).to(torch.bfloat16)
    s["out"].copy_(torch.where((s["slots"] >= 0)[:, None, None], out, s["out"]))
    spare[at] = new
    state.copy_(spare[:-1])
    return s["out"], state


SIZES = {"bf16": 2, "f32": 4, "e4m3": 1, "none": 0}


def work(case):
    if case["op"] == "norm":
        r, d = case["rows"], case["dim"]
        size = r * d * (SIZES[case["x"]] + 2 * SIZES[case["residual"]] + SIZES[case["out"]]) + 4 * d
        if case["out"] == "e4m3":
            size += 4 * r * -(-d // BLOCK)
        return dict(bytes=size, flops=6 * r * d)
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        kb, nb = -(-k // BLOCK), -(-n // BLOCK)
        size = m * k + n * k + 4 * (m * kb + nb * kb) + m * n * SIZES[case["out"]] + (4 * n if case["bias"] else 0)
        return dict(bytes=size, flops=2 * m * n * k)
    b, g, h, dk, dv = case["b"], case["g"], case["h"], case["dk"], case["dv"]
    gate = 4 * (h if case["gates"] == "head" else b * case.get("l", 1) * h)
    if case["op"] == "attention":
        rows = b * case["l"] / (2 if case["ragged"] else 1)  # lengths are spread evenly from none to all
        size = rows * (2 * g * dk + 2 * h * dv) * 2 + b * h * dk * dv * 4 * (2 if case["h0"] else 1) + gate
        # the recurrence itself: the state's update and its product with q
        return dict(bytes=size, flops=4 * rows * h * dk * dv)
    rows = b * (0.9 if case["slots"] else 1)
    return dict(bytes=rows * (8 * h * dk * dv + 4 * g * dk + 4 * h * dv) + gate, flops=5 * rows * h * dk * dv)


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        x = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        y = x / (x.square().sum(1, keepdim=True) / case["dim"] + EPS).sqrt() * s["weight"].double()
        got = [y]
        if case["out"] == "e4m3":
            # the definition's e4m3 values: three bits behind the first, at least 2^-9 apart
            kb = -(-case["dim"] // BLOCK)
            at = torch.arange(case["dim"], device=y.device) // BLOCK
            amax = torch.zeros(case["rows"], kb, dtype=y.dtype, device=y.device)
            amax.scatter_reduce_(1, at.expand_as(y), y.abs(), "amax")
            scales = (amax / E4M3_MAX).clamp_min(SCALE_MIN)
            t = y / scales[:, at]
            unit = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))) - 3)
            got = [torch.round(t / unit) * unit, scales]
        if s["residual"] is not None:
            got.append(x)
        return tuple(got) if len(got) > 1 else got[0]
    if case["op"] == "matmul":
        at = torch.arange(case["k"], device="cuda") // BLOCK
        a = s["a"].double().mul_(s["a_scales"].double()[:, at])
        rows = torch.arange(case["n"], device="cuda") // BLOCK
        w = s["w"].double().mul_(s["w_scales"].double()[rows][:, at])
        c = torch.einsum("mk,nk->mn", a, w)
        return c if s["bias"] is None else c.add_(s["bias"].double())
    b, h, g = case["b"], case["h"], case["g"]
    if case["op"] == "attention":
        l, dk, dv = case["l"], case["dk"], case["dv"]
        out = torch.zeros(b, l, h, dv, dtype=torch.float64, device="cuda")
        last = torch.zeros(b, h, dk, dv, dtype=torch.float64, device="cuda")
        for i in range(b):
            m = l if s["lengths"] is None else int(s["lengths"][i])
            gates = (s["log_decay"][i, :m] if case["gates"] == "token" else s["log_decay"].expand(m, h)).double()
            to = torch.cat([torch.zeros(1, h, dtype=torch.float64, device="cuda"), gates.cumsum(0)])
            for j in range(h):
                q, k, v = (s[x][i, :m, (j * g) // h if x != "v" else j].double() for x in "qkv")
                t = to[1:, j]
                start = torch.zeros(dk, dv, dtype=torch.float64, device="cuda") if s["h0"] is None else s["h0"][i, j].double()
                last[i, j] = start * to[m, j].exp() + k.t() @ (v * (to[m, j] - t).exp()[:, None])
                for r in range(0, m, 2048):
                    e = min(m, r + 2048)
                    seen = torch.arange(e, device="cuda")[None] <= torch.arange(r, e, device="cuda")[:, None]
                    d = (t[r:e, None] - t[None, :e]).masked_fill_(~seen, -math.inf).exp_()
                    d *= q[r:e] @ k[:e].t()
                    out[i, r:e, j] = (d @ v[:e] + (q[r:e] @ start) * t[r:e, None].exp()) * s["scale"]
        return out, last
    state = s["state"].double()
    out = torch.zeros(b, h, case["dv"], dtype=torch.float64, device="cuda")
    of = torch.arange(h, device="cuda") * g // h
    rows = torch.arange(b, device="cuda")
    at = rows if s["slots"] is None else s["slots"].long()
    rows, at = rows[at >= 0], at[at >= 0]
    gates = s["log_decay"].double().expand(b, h)[rows].exp()
    k, q, v = s["k"].double()[rows][:, of], s["q"].double()[rows][:, of], s["v"].double()[rows]
    state[at] = torch.einsum("bhkv,bh->bhkv", state[at], gates) + torch.einsum("bhk,bhv->bhkv", k, v)
    out[rows] = torch.einsum("bhk,bhkv->bhv", q, state[at]) * s["scale"]
    return out, state
