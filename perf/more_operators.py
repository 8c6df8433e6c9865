"""Cases of the operators that complete a quantized decoder block: the product of bf16
activations with packed 4-bit weights and its epilogue (bias, activation, gate, residual),
the norms of queries and keys with the position rotation and the writes to a key/value
cache, and attention over packed prompts and over a cache.

`own` selects who computes: the plain forms below (elementary torch operations in 32
bits, angles in 64), or the framework's entry points.
"""
import functools
import math

import torch

own = False

DEV = "cuda:0"
EPS = 1e-6
F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16
TYPES = {"bf16": BF16, "f32": F32}
SIZE = {"bf16": 2, "f32": 4}

# the most that a drawn case of each operator may cost (what the largest listed one does)
LINEAR_MOST = 8192 * 8192 * 57344
ROPE_MOST = 16384 * 80 * 128 * 4  # bytes
ATTN_MOST = 64 * 128 * (16384 * 16385 // 2)
CACHE_MOST = 1 << 28   # elements of one drawn cache


def listed():
    return [
        # one generated token through an output projection: bias, and the residual added
        {"name": "linear token 4096x4096", "op": "linear", "m": 1, "d_in": 4096, "d_out": 4096, "g": 128,
         "sym": False, "bias": True, "act": "none", "gated": False, "res": "bf16", "out": "bf16"},
        # sixteen sequences' next tokens through gate and up, their product on the way out
        {"name": "linear gate/up 16 tokens", "op": "linear", "m": 16, "d_in": 4096, "d_out": 22016, "g": 64,
         "sym": True, "bias": False, "act": "silu", "gated": True, "res": None, "out": "bf16"},
        # a short prompt through a down projection with an odd row count, added to an fp32 residual
        {"name": "linear down 515 tokens", "op": "linear", "m": 515, "d_in": 11008, "d_out": 4099, "g": 32,
         "sym": False, "bias": True, "act": "gelu", "gated": False, "res": "f32", "out": "f32"},
        # a prefill of four sequences through the largest layer's gate and up
        {"name": "linear gate/up 8192 tokens", "op": "linear", "m": 8192, "d_in": 8192, "d_out": 57344, "g": 128,
         "sym": False, "bias": False, "act": "silu", "gated": True, "res": None, "out": "bf16"},
        # one generated token, from the product's fp32 output into the cache
        {"name": "rope token", "op": "rope", "m": 1, "hq": 32, "hk": 8, "hd": 128, "rot": 128, "norm": True,
         "x": "f32", "pairs": False, "slots": True, "far": 100000},
        # a prompt of 4096 tokens into the cache
        {"name": "rope 4096 tokens", "op": "rope", "m": 4096, "hq": 32, "hk": 8, "hd": 128, "rot": 128, "norm": True,
         "x": "bf16", "pairs": False, "slots": True, "far": 0},
        # odd counts, a part of each head rotated in neighbouring pairs, no norm
        {"name": "rope odd, part of a head", "op": "rope", "m": 1003, "hq": 21, "hk": 3, "hd": 80, "rot": 32,
         "norm": False, "x": "f32", "pairs": True, "slots": False, "far": 1000},
        # calibration: eight sequences of a wide model
        {"name": "rope 16384 tokens", "op": "rope", "m": 16384, "hq": 64, "hk": 8, "hd": 128, "rot": 128, "norm": True,
         "x": "bf16", "pairs": False, "slots": False, "far": 0},
        # one sequence's next token over a cache: latency
        {"name": "attention token", "op": "attn", "b": 1, "q": 1, "past": 4095, "hq": 32, "hk": 8, "hd": 128,
         "causal": True},
        # the next tokens of 64 sequences, each with its own length
        {"name": "attention 64 tokens", "op": "attn", "b": 64, "q": 64, "past": 8192, "hq": 64, "hk": 8, "hd": 128,
         "causal": True},
        # seven prompts of different lengths in one pass, a head of keys for each of queries
        {"name": "attention 7 prompts", "op": "attn", "b": 7, "q": 8197, "past": 0, "hq": 32, "hk": 32, "hd": 128,
         "causal": True},
        # one long prompt of a wide model
        {"name": "attention 16384 tokens", "op": "attn", "b": 1, "q": 16384, "past": 0, "hq": 64, "hk": 8, "hd": 128,
         "causal": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, uniform over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["linear", "rope", "attn"])
    if op == "linear":
        g = rng.choice([32, 64, 128, -1])
        unit = max(g, 32)
        d_in = unit * max(1, _spread(rng, 256, 12288) // unit)
        gated = rng.random() < 0.4
        d_out = _spread(rng, 64, 16384) * (2 if gated else 1)
        m = _spread(rng, 1, min(8192, LINEAR_MOST // (d_in * d_out)))
        return {"op": op, "m": m, "d_in": d_in, "d_out": d_out, "g": g, "sym": rng.random() < 0.5,
                "bias": rng.random() < 0.5, "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu"] if gated else
                                                              ["none", "none", "silu", "gelu", "gelu_tanh", "relu"]),
                "gated": gated, "res": rng.choice([None, "bf16", "f32"]), "out": rng.choice(["bf16", "bf16", "f32"])}
    hd = rng.choice([64, 80, 96, 128, 128, 256])
    hk = rng.choice([1, 2, 3, 4, 8, 8, 16])
    hq = hk * rng.choice([1, 2, 4, 5, 8])
    if op == "rope":
        x = rng.choice(["bf16", "f32"])
        m = _spread(rng, 1, min(16384, ROPE_MOST // ((hq + 2 * hk) * hd * (SIZE[x] + 2))))
        return {"op": op, "m": m, "hq": hq, "hk": hk, "hd": hd, "rot": rng.choice([32, 64, hd, hd]),
                "norm": rng.random() < 0.7, "x": x, "pairs": rng.random() < 0.3,
                "slots": rng.random() < 0.5, "far": rng.choice([0, 0, 5000, 1000000])}
    if rng.random() < 0.5:  # the next tokens, one to four to a sequence, over a cache
        b = _spread(rng, 1, 128)
        q = b * rng.choice([1, 1, 1, 2, 4])
        past = _spread(rng, 16, min(65536, CACHE_MOST // (b * hk * hd)))
    else:                   # prompts, or pieces of prompts behind what the cache holds
        b = _spread(rng, 1, 16)
        past = rng.choice([0, 0, _spread(rng, 16, 8192)])
        q = max(b, _spread(rng, 64, 8192))
    c = {"op": op, "b": b, "q": q, "past": past, "hq": hq, "hk": hk, "hd": hd, "causal": rng.random() < 0.85}
    while _visible(c) * hq * hd > ATTN_MOST:
        c["q"] = max(b, c["q"] // 2 + 1)
    return c


# ------------------------------------------------------------------- inputs
def _lengths(c):
    """Queries and keys of each sequence: ragged, the same for every seed."""
    b, q = c["b"], c["q"]
    if q % b == 0 and q // b <= 4:
        lq = [q // b] * b
    else:
        weight = [3 + (5 * i + 2) % 7 for i in range(b)]
        lq = [1 + (q - b) * w // sum(weight) for w in weight]
        lq[-1] += q - sum(lq)
    past = [c["past"] - (i * 40503 % (c["past"] // 2 + 1)) for i in range(b)]
    return lq, [p + n for p, n in zip(past, lq)]


def _visible(c):
    """Pairs of a query and a key that it sees."""
    lq, lk = _lengths(c)
    if not c["causal"]:
        return sum(a * n for a, n in zip(lq, lk))
    return sum(a * (n - a) + a * (a + 1) // 2 for a, n in zip(lq, lk))


def _weights(c, gen):
    """Weights N(0, 0.02^2) with 0.1% of the entries ten times as large, on each group's 4-bit
    grid by rounding to nearest: packed codes (little-endian nibbles of 32-bit words), and the
    scales and zeros as binary16 bits."""
    d_out, d_in = c["d_out"], c["d_in"]
    G = d_in if c["g"] == -1 else c["g"]
    w = torch.randn((d_out, d_in), generator=gen, device=DEV).mul_(0.02)
    w *= 1.0 + 9.0 * (torch.rand((d_out, d_in), generator=gen, device=DEV) < 0.001)
    w = w.view(d_out, d_in // G, G)
    if c["sym"]:
        scale = (2.0 * w.abs().amax(2) / 15.0).half()
        zero = torch.full_like(scale, 8.0)
    else:
        lo, hi = w.amin(2).clamp(max=0.0), w.amax(2).clamp(min=0.0)
        scale = ((hi - lo) / 15.0).half()
        zero = (-lo / scale.float()).round().clamp(0.0, 15.0).half()
    q = (w / scale.float()[:, :, None]).round_().add_(zero.float()[:, :, None]).clamp_(0.0, 15.0).to(torch.int32)
    q = q.view(d_out, d_in // 8, 8) << torch.arange(0, 32, 4, device=DEV, dtype=torch.int32)
    words = q.sum(2, dtype=torch.int32)  # disjoint bits
    return words, scale.view(torch.int16), None if c["sym"] else zero.view(torch.int16)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "linear":
        m, n = c["m"], c["d_out"] // 2 if c["gated"] else c["d_out"]
        s["qw"], s["s16"], s["z16"] = _weights(c, gen)
        s["x"] = (_randn(gen, m, c["d_in"]) * _randn(gen, c["d_in"]).mul_(0.5).exp_()).to(BF16)
        s["bias"] = _randn(gen, c["d_out"]).to(BF16) if c["bias"] else None
        s["res"] = _randn(gen, m, n).mul_(2.0).to(TYPES[c["res"]]) if c["res"] else None
        s["y"] = torch.empty((m, n), dtype=TYPES[c["out"]], device=DEV)
        return s
    hq, hk, hd = c["hq"], c["hk"], c["hd"]
    if c["op"] == "rope":
        m = c["m"]
        # the stacked projections' output, some channels much larger than others
        x = (_randn(gen, m, hq + 2 * hk, hd) * _randn(gen, hq + 2 * hk, hd).mul_(0.7).exp_()).to(TYPES[c["x"]])
        s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        s["qn"] = s["kn"] = None
        if c["norm"]:
            s["qn"], s["kn"] = ((1.0 + 0.2 * _randn(gen, hd)).to(BF16) for _ in range(2))
        s["pos"] = torch.arange(m, device=DEV, dtype=torch.int32) + c["far"]
        s["freq"] = 500000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=F64) / c["rot"])
        rows = m
        s["slots"] = None
        if c["slots"]:  # the tokens' places among the pages of a cache
            rows = m + m // 2 + 64
            s["slots"] = torch.randperm(rows, generator=gen, device=DEV)[:m].contiguous()
        s["qo"] = torch.empty((m, hq, hd), dtype=BF16, device=DEV)
        s["ko"], s["vo"] = (_randn(gen, rows, hk, hd).to(BF16) for _ in range(2))
        return s
    lq, lk = _lengths(c)
    s["lq"], s["lk"] = lq, lk
    at = [0]
    for n in lq:
        at.append(at[-1] + n)
    s["cu_q"] = torch.tensor(at, dtype=torch.int32, device=DEV)
    if c["past"]:
        cap = max(lk) + 5
        order = [(7 * i + 3) % c["b"] if math.gcd(7, c["b"]) == 1 else i for i in range(c["b"])]
        s["start"] = [cap * o for o in order]
        s["kv_start"] = torch.tensor(s["start"], dtype=torch.int64, device=DEV)
        s["kv_len"] = torch.tensor(lk, dtype=torch.int32, device=DEV)
        rows = cap * c["b"]
    else:
        s["start"], s["kv_start"], s["kv_len"], rows = at[:-1], None, None, c["q"]
    # queries as a norm of each head leaves them; keys whose heads differ in scale; a tenth of
    # the keys close to some query's direction, so that the weights are not all alike
    s["q"] = _randn(gen, c["q"], hq, hd).mul_(1.5).to(BF16)
    kv = torch.empty((rows, 2, hk, hd), dtype=BF16, device=DEV)
    s["k"], s["v"] = kv[:, 0], kv[:, 1]
    for h in range(hk):
        kv[:, 0, h] = _randn(gen, rows, hd).mul_(0.5 + 0.5 * ((h * 3) % 4))
        kv[:, 1, h] = _randn(gen, rows, hd)
    near = torch.randint(0, rows, (max(1, rows // 10),), generator=gen, device=DEV)
    kv[near, 0] = s["q"][near % c["q"], ::hq // hk]
    s["out"] = torch.empty((c["q"], hq, hd), dtype=BF16, device=DEV)
    return s


@functools.lru_cache(maxsize=None)
def _entry_points():
    from post_weight_quantization_syrk_amd import gptq
    return gptq


def run(state):
    s, c = state, state["case"]
    if own:
        gptq = _entry_points()
        if c["op"] == "linear":
            return gptq.gptq_w4a16_linear(s["x"], s["qw"], s["s16"], s["z16"], group_size=c["g"], sym=c["sym"],
                                          bias=s["bias"], activation=c["act"], gated=c["gated"],
                                          residual=s["res"], out_dtype=TYPES[c["out"]], Y=s["y"])
        if c["op"] == "rope":
            q, k, v = gptq.gptq_qk_norm_rope(s["q"], s["k"], s["v"], positions=s["pos"], inv_freq=s["freq"],
                                             q_weight=s["qn"], k_weight=s["kn"], eps=EPS, interleaved=c["pairs"],
                                             slots=s["slots"], q_out=s["qo"], k_out=s["ko"], v_out=s["vo"])
            return {"q": q, "k": k, "v": v}
        return gptq.gptq_attention(s["q"], s["k"], s["v"], cu_q=s["cu_q"], kv_start=s["kv_start"],
                                   kv_len=s["kv_len"], causal=c["causal"], max_kv_len=max(s["lk"]), out=s["out"])
    if c["op"] == "linear":
        return _linear(s, c)
    if c["op"] == "rope":
        return _rope(s, c)
    return _attention(s, c)


# -------------------------------------------------------------- plain forms
def _activation(v, act):
    if act == "relu":
        return torch.where(v > 0.0, v, 0.0)
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _linear(s, c):
    q = (s["qw"][:, :, None] >> torch.arange(0, 32, 4, device=DEV, dtype=torch.int32)) & 15
    q = q.view(c["d_out"], s["s16"].shape[1], -1).to(F32)
    z = 8.0 if s["z16"] is None else s["z16"].view(torch.float16).to(F32)[:, :, None]
    w = ((q - z) * s["s16"].view(torch.float16).to(F32)[:, :, None]).view(c["d_out"], c["d_in"])
    y = s["x"].to(F32) @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"].to(F32)
    if c["gated"]:
        n = c["d_out"] // 2
        y = _activation(y[:, :n], c["act"]) * y[:, n:]
    else:
        y = _activation(y, c["act"])
    if s["res"] is not None:
        y = y + s["res"].to(F32)
    return y.to(TYPES[c["out"]])


def _rope(s, c):
    angle = s["pos"].to(F64)[:, None] * s["freq"][None, :]
    cos, sin = torch.cos(angle).to(F32)[:, None, :], torch.sin(angle).to(F32)[:, None, :]
    rot = c["rot"]

    def turned(x, weight):
        x = x.to(F32)
        if weight is not None:
            x = x / torch.sqrt((x * x).mean(2, keepdim=True) + EPS) * weight.to(F32)
        out = x.clone()
        if c["pairs"]:
            a, b = x[:, :, 0:rot:2], x[:, :, 1:rot:2]
            out[:, :, 0:rot:2], out[:, :, 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[:, :, :rot // 2], x[:, :, rot // 2:rot]
            out[:, :, :rot // 2], out[:, :, rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        return out.to(BF16)

    q, k, v = turned(s["q"], s["qn"]), turned(s["k"], s["kn"]), s["v"].to(BF16)
    if s["slots"] is None:
        return {"q": q, "k": k, "v": v}
    s["ko"][s["slots"]] = k
    s["vo"][s["slots"]] = v
    return {"q": q, "k": s["ko"], "v": s["vo"]}


def _attention(s, c):
    hq, hk, hd = c["hq"], c["hk"], c["hd"]
    g = hq // hk
    out = torch.empty((c["q"], hq, hd), dtype=BF16, device=DEV)
    q0 = 0
    for lq, lk, k0 in zip(s["lq"], s["lk"], s["start"]):
        hidden = None
        if c["causal"] and lq > 1:
            hidden = torch.arange(lk, device=DEV)[None, :] > torch.arange(lq, device=DEV)[:, None] + (lk - lq)
        k = s["k"][k0:k0 + lk].to(F32).permute(1, 2, 0)    # [hk, hd, lk]
        v = s["v"][k0:k0 + lk].to(F32).transpose(0, 1)     # [hk, lk, hd]
        q = s["q"][q0:q0 + lq].to(F32).view(lq, hk, g, hd).permute(1, 2, 0, 3)  # [hk, g, lq, hd]
        step = max(1, (1 << 29) // (lq * lk))              # heads whose scores take 2 GB
        if step >= g:                                      # whole groups at once
            per = step // g
            pieces = [(slice(h, h + per), slice(0, g)) for h in range(0, hk, per)]
        else:
            pieces = [(slice(h, h + 1), slice(i, i + step)) for h in range(hk) for i in range(0, g, step)]
        for hs, gs in pieces:
            p = q[hs, gs] @ k[hs][:, None] * hd ** -0.5
            if hidden is not None:
                p.masked_fill_(hidden, -math.inf)
            p = torch.exp(p - p.amax(3, keepdim=True))
            o = (p @ v[hs][:, None]) / p.sum(3, keepdim=True)
            out.view(c["q"], hk, g, hd)[q0:q0 + lq, hs, gs] = o.permute(2, 0, 1, 3).to(BF16)
        q0 += lq
    return out


# --------------------------------------------------------- exact, in 64 bits
def exact(case, seed):
    s, c = prepare(case, seed), case
    return {"linear": _exact_linear, "rope": _exact_rope, "attn": _exact_attention}[c["op"]](s, c)


def _exact_linear(s, c):
    G = c["d_in"] if c["g"] == -1 else c["g"]
    x = s["x"].to(F64)
    n = c["d_out"] // 2 if c["gated"] else c["d_out"]

    def product(lo, hi):
        """The columns lo..hi - 1 of X W^T + bias."""
        cols = []
        for a in range(lo, hi, 4096):
            b = min(hi, a + 4096)
            nib = [((s["qw"][a:b].to(torch.int64) >> (4 * k)) & 15) for k in range(8)]
            w = torch.stack(nib, dim=2).reshape(b - a, c["d_in"]).to(F64)
            w -= 8.0 if c["sym"] else s["z16"][a:b].view(torch.float16).to(F64).repeat_interleave(G, dim=1)
            w *= s["s16"][a:b].view(torch.float16).to(F64).repeat_interleave(G, dim=1)
            y = torch.matmul(x, w.t())
            cols.append(y if s["bias"] is None else y + s["bias"][a:b].to(F64))
        return torch.cat(cols, dim=1)

    y = product(0, n)
    if c["act"] == "relu":
        y = y.clamp(min=0.0)
    elif c["act"] == "silu":
        y = y * torch.special.expit(y)
    elif c["act"] == "gelu":
        y = y * torch.special.ndtr(y)
    elif c["act"] == "gelu_tanh":
        y = y * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3))
    if c["gated"]:
        y = y * product(n, 2 * n)
    return y if s["res"] is None else y + s["res"].to(F64)


def _exact_rope(s, c):
    half = c["rot"] // 2
    turn = torch.polar(torch.ones((), dtype=F64, device=DEV),
                       torch.outer(s["pos"].to(F64), s["freq"]))[:, None, :]  # e^(i angle)

    def turned(x, weight):
        x = x.to(F64)
        if weight is not None:
            x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / c["hd"] + EPS) * weight.to(F64)
        first, rest = x[..., :2 * half], x[..., 2 * half:]
        if c["pairs"]:
            z = torch.view_as_complex(first.unflatten(-1, (half, 2)).contiguous()) * turn
            return torch.cat([torch.view_as_real(z).flatten(-2), rest], dim=-1)
        z = torch.complex(first[..., :half].contiguous(), first[..., half:].contiguous()) * turn
        return torch.cat([z.real, z.imag, rest], dim=-1)

    q, k, v = turned(s["q"], s["qn"]), turned(s["k"], s["kn"]), s["v"].to(F64)
    if s["slots"] is not None:
        k = s["ko"].to(F64).index_copy(0, s["slots"], k)
        v = s["vo"].to(F64).index_copy(0, s["slots"], v)
    return {"q": q, "k": k, "v": v}


def _exact_attention(s, c):
    g = c["hq"] // c["hk"]
    out = torch.empty((c["q"], c["hq"], c["hd"]), dtype=F64, device=DEV)
    q0 = 0
    for lq, lk, k0 in zip(s["lq"], s["lk"], s["start"]):
        rows = max(1, (1 << 27) // (g * lk))
        for h in range(c["hk"]):
            k, v = s["k"][k0:k0 + lk, h].to(F64), s["v"][k0:k0 + lk, h].to(F64)
            for a in range(0, lq, rows):
                b = min(lq, a + rows)
                seen = lk - lq + b if c["causal"] else lk   # the last of these queries sees so many keys
                q = s["q"][q0 + a:q0 + b, h * g:(h + 1) * g].to(F64)
                score = torch.tensordot(q, k[:seen], dims=([2], [1])) / math.sqrt(c["hd"])
                if c["causal"]:
                    i = torch.arange(a, b, device=DEV)[:, None]
                    blind = torch.arange(seen, device=DEV)[None, :] - i > lk - lq
                    score = torch.where(blind[:, None, :], -math.inf, score)
                weight = torch.exp(score - torch.logsumexp(score, dim=2, keepdim=True))
                out[q0 + a:q0 + b, h * g:(h + 1) * g] = torch.tensordot(weight, v[:seen], dims=([2], [0]))
        q0 += lq
    return out


# ------------------------------------------------------------- what it takes
def work(case):
    c = case
    if c["op"] == "linear":
        m, n = c["m"], c["d_out"] // 2 if c["gated"] else c["d_out"]
        ng = 1 if c["g"] == -1 else c["d_in"] // c["g"]
        b = c["d_out"] * (c["d_in"] // 2 + ng * (2 if c["sym"] else 4)) + 2 * m * c["d_in"]
        b += (2 * c["d_out"] if c["bias"] else 0) + m * n * ((SIZE[c["res"]] if c["res"] else 0) + SIZE[c["out"]])
        return {"bytes": b, "flops": 2 * m * c["d_in"] * c["d_out"]}
    heads = c["hq"] + 2 * c["hk"]
    if c["op"] == "rope":
        m = c["m"]
        return {"bytes": m * heads * c["hd"] * (SIZE[c["x"]] + 2) + m * (12 if c["slots"] else 4) + 4 * c["rot"],
                "flops": m * (c["hq"] + c["hk"]) * (3 * c["rot"] + (5 * c["hd"] if c["norm"] else 0))}
    _, lk = _lengths(c)
    return {"bytes": 4 * c["q"] * c["hq"] * c["hd"] + 4 * sum(lk) * c["hk"] * c["hd"],
            "flops": 4 * c["hd"] * c["hq"] * _visible(c)}
