"""Cases of the operators that run a quantized layer: the residual addition with the
root-mean-square norm and its 8-bit output, the product of 4-bit weights with a few
tokens (bf16), and the product of 4-bit weights with 8-bit activations.

`own` selects who computes: the plain forms below (elementary torch operations in 32
bits), or the framework's entry points.
"""
import functools
import math

import torch

own = False

DEV = "cuda:0"
EPS = 1e-5
F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16
TYPES = {"bf16": BF16, "f32": F32, "i8": torch.int8}
SIZE = {"bf16": 2, "f32": 4, "i8": 1}

# the most that a drawn case of each operator may cost (what the largest listed one does)
NORM_MOST = 16384 * 8192
VEC_MOST = 28672 * 8192
MUL_MOST = 8192 * 28672 * 8192


def listed():
    return [
        # one generated token: a product's fp32 output is added to the bf16 residual, and
        # the normalized row goes on in 8 bits
        {"name": "norm token i8", "op": "norm", "m": 1, "d": 4096, "x": "f32", "r": "bf16", "out": "i8", "pad": 0},
        # two sequences of 2048 tokens on their way to an 8-bit product
        {"name": "norm 4096 tokens i8", "op": "norm", "m": 4096, "d": 4096, "x": "bf16", "r": "bf16", "out": "i8", "pad": 0},
        # odd width, everything in fp32: no row but the first is aligned
        {"name": "norm odd f32 i8", "op": "norm", "m": 1000, "d": 5003, "x": "f32", "r": "f32", "out": "i8", "pad": 0},
        # calibration or prefill of eight sequences of a wide model, bf16 throughout
        {"name": "norm 16384 tokens bf16", "op": "norm", "m": 16384, "d": 8192, "x": "bf16", "r": "bf16", "out": "bf16", "pad": 0},
        # the smallest layer, one token: the call's latency
        {"name": "vec 256x256", "op": "vec", "m": 1, "d_in": 256, "d_out": 256, "g": 128, "sym": False},
        # one token through an attention projection
        {"name": "vec 4096x4096", "op": "vec", "m": 1, "d_in": 4096, "d_out": 4096, "g": 128, "sym": False},
        # sixteen sequences' next tokens through a gate or up projection
        {"name": "vec gate 16 tokens", "op": "vec", "m": 16, "d_in": 4096, "d_out": 11008, "g": 64, "sym": True},
        # one token through the largest layer, one group per row
        {"name": "vec 28672x8192", "op": "vec", "m": 1, "d_in": 8192, "d_out": 28672, "g": -1, "sym": False},
        # one token in 8 bits through an attention projection
        {"name": "mul token 4096x4096", "op": "mul", "m": 1, "d_in": 4096, "d_out": 4096, "g": 128, "sym": False},
        # a ragged batch of next tokens through a down projection with an odd row count
        {"name": "mul down 37 tokens", "op": "mul", "m": 37, "d_in": 11008, "d_out": 4099, "g": 32, "sym": False},
        # a short prompt through a gate or up projection
        {"name": "mul gate 515 tokens", "op": "mul", "m": 515, "d_in": 4096, "d_out": 11008, "g": 64, "sym": True},
        # a prefill of four sequences through the largest layer
        {"name": "mul 8192 tokens", "op": "mul", "m": 8192, "d_in": 8192, "d_out": 28672, "g": 128, "sym": False},
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, uniform over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm", "vec", "mul"])
    if op == "norm":
        d = _spread(rng, 256, 12288)
        d = d | 1 if rng.random() < 0.3 else (d + 7) // 8 * 8
        m = _spread(rng, 1, min(16384, NORM_MOST // d))
        return {"op": op, "m": m, "d": d, "x": rng.choice(["bf16", "f32"]), "r": rng.choice(["bf16", "f32"]),
                "out": rng.choice(["bf16", "i8"]), "pad": rng.choice([0, 0, 8, 24])}
    g = rng.choice([32, 64, 128, -1])
    unit = max(g, 32)
    d_in = unit * max(1, _spread(rng, 256, 12288) // unit)
    d_out = _spread(rng, 64, min(32768, VEC_MOST // d_in))
    m = _spread(rng, 1, 64) if op == "vec" else _spread(rng, 1, min(8192, MUL_MOST // (d_in * d_out)))
    return {"op": op, "m": m, "d_in": d_in, "d_out": d_out, "g": g, "sym": rng.random() < 0.5}


def _activations(m, d, gen):
    """N(0, 1) entries times a log-normal(0, 1) scale per channel, fp32."""
    return torch.randn((m, d), generator=gen, device=DEV) * torch.randn(d, generator=gen, device=DEV).exp()


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


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    m = c["m"]
    if c["op"] == "norm":
        d, ld = c["d"], c["d"] + c["pad"]
        x = torch.zeros((m, ld), dtype=TYPES[c["x"]], device=DEV)[:, :d]
        x.copy_(0.3 * _activations(m, d, gen))
        r = torch.zeros((m, ld), dtype=TYPES[c["r"]], device=DEV)[:, :d]
        r.copy_(_activations(m, d, gen))
        s["x"], s["r"] = x, r
        s["w"] = (1.0 + 0.2 * torch.randn(d, generator=gen, device=DEV)).to(BF16)
        s["out"] = torch.empty((m, d), dtype=TYPES[c["out"]], device=DEV)
        s["r_out"] = torch.empty((m, d), dtype=TYPES[c["r"]], device=DEV)
        s["scales"] = torch.empty(m, dtype=F32, device=DEV) if c["out"] == "i8" else None
        return s
    s["qw"], s["s16"], s["z16"] = _weights(c, gen)
    x = _activations(m, c["d_in"], gen)
    if c["op"] == "vec":
        s["x"] = x.to(BF16)
    else:
        s["xs"] = x.abs().amax(1) / 127.0
        s["x"] = (x / s["xs"][:, None]).round().clamp(-127.0, 127.0).to(torch.int8)
    s["y"] = torch.empty((m, c["d_out"]), dtype=F32, device=DEV)
    return s


@functools.lru_cache(maxsize=None)
def _entry_points():
    from post_weight_quantization_syrk_amd import gptq
    return gptq


def run(state):
    s, c = state, state["case"]
    if own:
        gptq = _entry_points()
        if c["op"] == "norm":
            out, scales, r = gptq.gptq_add_rmsnorm(s["x"], s["w"], residual=s["r"], residual_out=s["r_out"],
                                                   eps=EPS, out_dtype=TYPES[c["out"]], out=s["out"],
                                                   out_scales=s["scales"])
            if c["out"] == "i8":
                return {"out": out * scales[:, None], "scales": scales, "residual": r}
            return {"out": out, "residual": r}
        if c["op"] == "vec":
            return gptq.gptq_w4a16_matvec(s["x"], s["qw"], s["s16"], s["z16"], group_size=c["g"],
                                          sym=c["sym"], Y=s["y"])
        return gptq.gptq_w4a8_matmul(s["x"], s["xs"], s["qw"], s["s16"], s["z16"], group_size=c["g"],
                                     sym=c["sym"], Y=s["y"])
    if c["op"] == "norm":
        return _norm(s["x"], s["r"], s["w"], c["out"])
    x = s["x"].to(F32)
    if c["op"] == "mul":
        x = x * s["xs"][:, None]
    return x @ _dequantized(s["qw"], s["s16"], s["z16"]).t()


def _norm(x, r, w, out):
    """The residual's addition, the norm, and its output in bf16 or in 8 bits with one scale
    per row.  The quotients that decide an 8-bit code are formed in 64 bits: in 32 the ones
    next to a border fall to either side."""
    h = (x.to(F32) + r.to(F32)).to(r.dtype)
    hf = h.to(F32)
    rstd = 1.0 / torch.sqrt((hf * hf).mean(1, keepdim=True) + EPS)
    if out == "bf16":
        return {"out": (hf * rstd * w.to(F32)).to(BF16), "residual": h}
    p = h.to(F64) * w.to(F64)
    top = p.abs().amax(1, keepdim=True)
    scale = (top * rstd.to(F64) / 127.0).to(F32)
    empty = scale == 0.0
    codes = torch.where(empty, 0.0, torch.round(127.0 * p / top))
    scale = torch.where(empty, 1.0, scale)
    return {"out": codes.to(F32) * scale, "scales": scale[:, 0], "residual": h}


def _dequantized(qw, s16, z16):
    """W_hat = s (q - z), fp32."""
    d_out, words = qw.shape
    q = (qw[:, :, None] >> torch.arange(0, 32, 4, device=qw.device, dtype=torch.int32)) & 15
    q = q.view(d_out, s16.shape[1], -1).to(F32)
    z = 8.0 if z16 is None else z16.view(torch.float16).to(F32)[:, :, None]
    return ((q - z) * s16.view(torch.float16).to(F32)[:, :, None]).view(d_out, 8 * words)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "norm":
        r, w = s["r"].to(F64), s["w"].to(F64)
        h = (s["x"].to(F64) + r).to(s["r"].dtype)
        v = h.to(F64)
        y = v * w / (v.square().mean(dim=1) + EPS).sqrt()[:, None]
        if c["out"] == "bf16":
            return {"out": y, "residual": v}
        p = v * w
        top = p.abs().max(dim=1).values
        scale = y.abs().max(dim=1).values / 127.0
        return {"out": torch.round(127.0 * p / top[:, None]) * scale[:, None], "scales": scale, "residual": v}
    nib = [((s["qw"].to(torch.int64) >> (4 * k)) & 15) for k in range(8)]
    q = torch.stack(nib, dim=2).reshape(c["d_out"], c["d_in"]).to(F64)
    G = c["d_in"] if c["g"] == -1 else c["g"]
    scale = s["s16"].view(torch.float16).to(F64).repeat_interleave(G, dim=1)
    if c["sym"]:
        q -= 8.0
    else:
        q -= s["z16"].view(torch.float16).to(F64).repeat_interleave(G, dim=1)
    q *= scale
    y = torch.matmul(s["x"].to(F64), q.t())
    return y * s["xs"].to(F64)[:, None] if c["op"] == "mul" else y


def work(case):
    c = case
    if c["op"] == "norm":
        per = SIZE[c["x"]] + 2 * SIZE[c["r"]] + SIZE[c["out"]]
        return {"bytes": c["m"] * c["d"] * per + 2 * c["d"] + (4 * c["m"] if c["out"] == "i8" else 0),
                "flops": 6 * c["m"] * c["d"]}
    ng = 1 if c["g"] == -1 else c["d_in"] // c["g"]
    weights = c["d_out"] * (c["d_in"] // 2 + ng * (2 if c["sym"] else 4))
    x = c["m"] * (c["d_in"] * (2 if c["op"] == "vec" else 1) + (4 if c["op"] == "mul" else 0))
    return {"bytes": weights + x + 4 * c["m"] * c["d_out"], "flops": 2 * c["m"] * c["d_in"] * c["d_out"]}
