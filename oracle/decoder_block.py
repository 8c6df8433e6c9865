"""What stands between and behind the quantized products of a decoder block, float64
reference: the products' epilogue, the norms of queries and keys with the rotation, and
attention over packed sequences.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activate(v, kind: str) -> np.ndarray:
    v = np.asarray(v, dtype=np.float64)
    if kind == "none":
        return v
    if kind == "relu":
        return np.maximum(v, 0.0)
    if kind == "silu":
        return v * 0.5 * (1.0 + np.tanh(0.5 * v))
    if kind == "gelu":
        return 0.5 * v * (1.0 + _erf(v / math.sqrt(2.0)))
    if kind == "gelu_tanh":
        return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    raise ValueError(kind)


def epilogue(v, kind: str, gated: bool, residual=None) -> np.ndarray:
    """act(v) + residual, or, gated, act(first half of v's columns) times the second half."""
    if gated:
        n = v.shape[1] // 2
        y = activate(v[:, :n], kind) * v[:, n:]
    else:
        y = activate(v, kind)
    return y if residual is None else y + residual


def norm_rope(x, weight, positions, inv_freq, *, eps: float, interleaved: bool) -> np.ndarray:
    """x [m, heads, hd]: normalized over each head (weight None: not), then the first 2
    len(inv_freq) columns turned pair by pair."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt(np.mean(y * y, axis=2, keepdims=True) + eps) * np.asarray(weight, np.float64)
    out = y.copy()
    half = 0 if inv_freq is None else len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        angle = np.asarray(positions, np.float64) * float(inv_freq[i])
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        out[:, :, a] = y[:, :, a] * c - y[:, :, b] * s
        out[:, :, b] = y[:, :, b] * c + y[:, :, a] * s
    return out


def attention_weights(q, k, scale: float, causal: bool):
    """Weights [lq, lk] of one head: softmax over the keys that each query sees, zeros where it
    sees none; and which it sees."""
    lq, lk = q.shape[0], k.shape[0]
    seen = np.ones((lq, lk), dtype=bool)
    if causal:
        seen = np.arange(lk)[None, :] <= np.arange(lq)[:, None] + (lk - lq)
    with np.errstate(invalid="ignore"):
        score = np.where(seen, (np.asarray(q, np.float64) @ np.asarray(k, np.float64).T) * scale, -np.inf)
    top = np.max(score, axis=1, initial=-np.inf, keepdims=True)
    w = np.where(seen, np.exp(score - np.where(np.isfinite(top), top, 0.0)), 0.0)
    total = w.sum(axis=1, keepdims=True)
    return w / np.where(total > 0.0, total, 1.0), seen


def attention(q, k, v, cu_q, starts, lens, *, scale: float, causal: bool) -> np.ndarray:
    """q [tq, hq, hd], k and v [rows, hk, hd]; rows of the result outside all sequences are NaN."""
    tq, hq, hd = q.shape
    group = hq // k.shape[1]
    out = np.full((tq, hq, hd), np.nan)
    for s in range(len(cu_q) - 1):
        a, b, k0, n = cu_q[s], cu_q[s + 1], starts[s], lens[s]
        for h in range(hq):
            w, _ = attention_weights(q[a:b, h], k[k0:k0 + n, h // group], scale, causal)
            out[a:b, h] = w @ np.asarray(v[k0:k0 + n, h // group], np.float64)
    return out
