"""Pins of the norm oracle (residual sum, root-mean-square norm, 8-bit codes).  CPU only."""
from __future__ import annotations

from fractions import Fraction

import numpy as np
import torch

import oracle


def test_residual_sum_rounds_as_torch_does():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((64, 33)) * np.exp(4 * rng.standard_normal((64, 33)))).astype(np.float32)
    r = oracle.round_bf16(rng.standard_normal((64, 33)).astype(np.float32))
    want = (torch.from_numpy(x) + torch.from_numpy(r)).bfloat16().float().numpy()
    np.testing.assert_array_equal(oracle.residual_sum(x, r, "bf16"), want)
    np.testing.assert_array_equal(oracle.residual_sum(x, r, "f32"), x + r)
    np.testing.assert_array_equal(oracle.residual_sum(x, None, "bf16"), x)


def test_hand_example():
    # h = (3, 4): mean square 12.5, eps 12.5: divided by 5; weights (5, 10): y = (3, 8)
    h = np.array([[3.0, 4.0]], dtype=np.float32)
    w = np.array([5.0, 10.0])
    np.testing.assert_allclose(oracle.rms_norm(h, w, 12.5), [[3.0, 8.0]], rtol=1e-15)
    q, s = oracle.norm_codes(h, w, 12.5)
    np.testing.assert_array_equal(q, [[48, 127]])  # 127 * 15 / 40 = 47.625
    np.testing.assert_allclose(s, [8.0 / 127.0], rtol=1e-15)


def test_codes_against_exact_fractions():
    # rint of the exact quotient, ties to even, for bf16 inputs (whose products are short)
    rng = np.random.default_rng(3)
    h = oracle.round_bf16(rng.standard_normal((6, 40)).astype(np.float32))
    w = oracle.round_bf16(1 + 0.2 * rng.standard_normal(40).astype(np.float32))
    h[0, :8] = np.arange(8)   # whole numbers: ties
    h[0, 8:] = 254.0
    q, _ = oracle.norm_codes(h, w, 1e-6)
    for i in range(6):
        p = [Fraction(float(a)) * Fraction(float(b)) for a, b in zip(h[i], w)]
        top = max(abs(v) for v in p)
        np.testing.assert_array_equal(q[i], [round(127 * v / top) for v in p])


def test_planted_mistakes_fail():
    rng = np.random.default_rng(5)
    h = rng.standard_normal((3, 50)).astype(np.float32)
    w = 1 + 0.3 * rng.standard_normal(50)
    q, s = oracle.norm_codes(h, w, 1e-6)
    y = oracle.rms_norm(h, w, 1e-6)
    assert np.max(np.abs(s[:, None] * q - y)) <= 0.5 * s.max() * (1 + 1e-12)
    without_weight = np.rint(127 * h / np.abs(h).max(1, keepdims=True))
    assert (without_weight != q).any()
    truncated = np.trunc(y / s[:, None])
    assert np.max(np.abs(s[:, None] * truncated - y)) > 0.5 * s.max()


def test_empty_rows():
    h = np.zeros((2, 5), dtype=np.float32)
    h[1, 2] = 1e-30
    q, s = oracle.norm_codes(h, np.ones(5), 1e30)
    np.testing.assert_array_equal(q, np.zeros((2, 5)))
    np.testing.assert_array_equal(s, [1.0, 1.0])
    np.testing.assert_array_equal(oracle.rms_norm(np.zeros((1, 4)), np.ones(4), 0.0), np.zeros((1, 4)))
