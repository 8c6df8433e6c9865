"""Bars and inputs shared by the tests of the calls that complete a decoder block."""
from __future__ import annotations

import numpy as np
import torch

import oracle
from post_weight_quantization_syrk_amd import synth
from serve_util import DEV, U16, U32, abs_terms, packed_weights

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": U16, "f32": U32}


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def randn(rng, *shape):
    return rng.standard_normal(shape, dtype=np.float32)


def device(a, kind):
    """A float32 array on the GPU in its type, and the values it then has in float64."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV).to(TORCH[kind])
    return t, f64(t)


def padded(t, pad, fill=float("nan")):
    """t's rows inside rows that are `pad` longer, the rest NaN."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


# ------------------------------------------------------------------ linear
def linear_reference(x64, qw, s16, z16, g, sym, bias, act, gated, residual, out):
    """(value, bound) of Y, float64.

    Sums: products are exact (bf16 times q or q - z, whole numbers up to 15 in
    magnitude), a group's K-term fp32 sums are off by at most K u times the sum of
    their terms' magnitudes, and conversions, joins with the zero, scaling and the
    addition of groups, runs and splits round at most 8 + K / 32 times more (K / 32
    groups at most, each added once); s (q + z) covers q - z and its parts.
    Activation: every one here has slopes below 1.13 in magnitude, and its own
    evaluation is off by at most 40 u |act| + 8 u (expf and erfcf within 16 u, the
    roundings of their arguments: for gelu 2.83 x^3 erfc(x) u < u, for the logistic
    forms 4 u v u'(v) s (1 - s) < 8 u).  Gate, residual and output: one rounding each.
    """
    K = x64.shape[1]
    v = oracle.dequant_matmul(x64, qw, s16, z16, bits=4, group_size=g, sym=sym)
    ev = (K + K / 32 + 8) * U32 * (np.abs(x64) @ abs_terms(qw, s16, z16, sym, g, K).T)
    if bias is not None:
        v = v + bias
        ev = ev + U32 * (np.abs(v) + ev)
    n = v.shape[1] // 2 if gated else v.shape[1]
    a = oracle.activate(v[:, :n], act)
    ea = ev[:, :n] if act == "none" else 1.13 * ev[:, :n] + 40 * U32 * np.abs(a) + 8 * U32
    if gated:
        b, eb = v[:, n:], ev[:, n:]
        y = a * b
        ey = np.abs(a) * eb + np.abs(b) * ea + ea * eb
        ey = ey + U32 * (np.abs(y) + ey)
    else:
        y, ey = a, ea
    if residual is not None:
        y = y + residual
        ey = ey + U32 * (np.abs(y) + ey)
    return y, ey + HALF_STEP[out] * (np.abs(y) + ey) + 1e-38


def weights(d_in, d_out, g, sym, seed):
    _, qw, s16, z16 = packed_weights(d_in, d_out, g, seed)
    return qw, s16, None if sym else z16


# -------------------------------------------------------------------- rope
def rope_reference(x64, weight, positions, inv_freq, eps, interleaved):
    """(value, bound) of norm_rope's bf16 output, float64.

    rstd: a sum of hd squares, all of one sign, is off by (hd + 1) u relative, its
    root by half of that, with the quotient, eps, root and reciprocal four more.
    cos, sin: the angle (float64, three roundings of 2^-53 of it) loses its turns
    exactly and is then rounded once to float32 (pi u), the functions are within 4 u.
    Two products and their sum: 3 u of |a| + |b|.  Output: half a step of bf16."""
    m, heads, hd = x64.shape
    y = oracle.norm_rope(x64, weight, positions, inv_freq, eps=eps, interleaved=interleaved)
    n = oracle.norm_rope(x64, weight, None, None, eps=eps, interleaved=interleaved)
    size = np.abs(n)
    bound = np.zeros_like(size) if weight is None else (hd / 2 + 8) * U32 * size
    half = 0 if inv_freq is None else len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        both = (size[:, :, a] + size[:, :, b])
        angle = np.abs(np.asarray(positions, np.float64) * inv_freq[i])[:, None]
        e = (bound[:, :, a] + bound[:, :, b]) + both * ((4 + 4 + 3) * U32 + 3 * 2.0 ** -53 * angle)
        bound[:, :, a], bound[:, :, b] = e, e
    return y, bound + U16 * (np.abs(y) + bound) + 1e-38


# --------------------------------------------------------------- attention
def attention_reference(q, k, v, cu_q, starts, lens, scale, causal):
    """(value, bound) of the bf16 output, float64; NaN outside all sequences.

    A score is an hd-term fp32 sum of exact products: off by hd u sum |q||k|.  The
    weight's exponent, s c - m c in log2 units, adds 4 u (|s c| + |m c|), exp2 4 u,
    and bf16 half a step: delta_j relative in all.  Numerator and denominator use the
    same rounded weights, so the quotient moves by at most sum w_j delta_j (|v_j| +
    |out|), and fp32 sums over lk keys, rescalings and the joins of waves and splits
    by (2 lk + 64) u of the same."""
    tq, hq, hd = q.shape
    group = hq // k.shape[1]
    out, bound = np.full((tq, hq, hd), np.nan), np.full((tq, hq, hd), np.nan)
    for s in range(len(cu_q) - 1):
        a, b, k0, n = cu_q[s], cu_q[s + 1], starts[s], lens[s]
        for h in range(hq):
            kk, vv = k[k0:k0 + n, h // group], v[k0:k0 + n, h // group]
            w, _ = oracle.attention_weights(q[a:b, h], kk, scale, causal)
            o = w @ vv
            size = np.abs(q[a:b, h]) @ np.abs(kk).T * scale
            most = size.max(axis=1, initial=0.0)[:, None]
            delta = (hd + 8) * U32 * size + 8 * U32 * most + 4 * U32 + U16 * (1 + 2.0 ** -7)
            e = (w * delta) @ np.abs(vv) + (w * delta).sum(1, keepdims=True) * np.abs(o)
            e += (2 * n + 64) * U32 * (w @ np.abs(vv) + np.abs(o))
            out[a:b, h], bound[a:b, h] = o, 1.05 * e + U16 * (np.abs(o) + e) + 1e-38
    return out, bound


def within(got, value, bound, what=""):
    err = np.abs(f64(got) - value)
    worst = float(np.max(err / np.maximum(bound, 1e-300), initial=0.0))
    print(f"{what} max err / bound {worst:.3f}", flush=True)
    assert np.all(err <= bound), (what, worst)
