"""Residual addition, root-mean-square norm and 8-bit codes, float64 reference.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The affine grid of "GPTQ：基于近似二阶信息的大模型权重量化", 对称与仿射量化, in its
symmetric form on one row of activations: scale = max|y| / 127, q = rint(y /
scale).  With y_c = p_c rstd and p_c = h_c w_c the factor rstd > 0 cancels, q_c
= rint(127 p_c / max|p|), and p is exact in float64 for float32 h and w.
"""
from __future__ import annotations

import numpy as np


def round_bf16(a) -> np.ndarray:
    """float32 values rounded to bfloat16 (nearest, ties to even), as float32."""
    u = np.ascontiguousarray(a, dtype=np.float32).view(np.uint32)
    u = (u + ((u >> np.uint32(16)) & np.uint32(1)) + np.uint32(0x7FFF)) & np.uint32(0xFFFF0000)
    return u.view(np.float32)


def residual_sum(x, r, r_dtype: str) -> np.ndarray:
    """h = x + r rounded to float32 and then to r's type; x itself without r."""
    if r is None:
        return np.asarray(x, dtype=np.float32)
    h = np.asarray(x, dtype=np.float32) + np.asarray(r, dtype=np.float32)
    return round_bf16(h) if r_dtype == "bf16" else h


def rms_norm(h, weight, eps: float) -> np.ndarray:
    """y [m, d] float64."""
    h = np.asarray(h, dtype=np.float64)
    ms = np.mean(h * h, axis=1) + eps
    rstd = np.where(ms > 0.0, 1.0 / np.sqrt(np.where(ms > 0.0, ms, 1.0)), 0.0)
    return h * np.asarray(weight, dtype=np.float64) * rstd[:, None]


def norm_codes(h, weight, eps: float):
    """(codes int8 [m, d], scale float64 [m] before its rounding to float32; 1 for an empty row)."""
    p = np.asarray(h, dtype=np.float64) * np.asarray(weight, dtype=np.float64)
    top = np.max(np.abs(p), axis=1)
    scale = np.max(np.abs(rms_norm(h, weight, eps)), axis=1) / 127.0
    empty = np.asarray(scale, dtype=np.float32) == 0.0
    q = np.rint(127.0 * p / np.where(empty, 1.0, top)[:, None])
    return (np.where(empty[:, None], 0.0, q).astype(np.int8), np.where(empty, 1.0, scale))
