"""Pins of the decoder block's reference: values worked by hand and identities that hold for
any input; a planted mistake fails them."""
from __future__ import annotations

import math

import numpy as np
import pytest

import oracle


def test_activations_at_known_points():
    v = np.array([-30.0, -1.0, 0.0, 1.0, 30.0])
    np.testing.assert_array_equal(oracle.activate(v, "none"), v)
    np.testing.assert_array_equal(oracle.activate(v, "relu"), [0, 0, 0, 1, 30])
    s = 1.0 / (1.0 + math.exp(-1.0))
    np.testing.assert_allclose(oracle.activate(v, "silu")[1:], [-(1 - s), 0, s, 30], rtol=1e-12)
    phi = 0.5 * (1.0 + math.erf(math.sqrt(0.5)))
    np.testing.assert_allclose(oracle.activate(v, "gelu")[1:], [-(1 - phi), 0, phi, 30], rtol=1e-12)
    t = 0.5 * (1.0 + math.tanh(math.sqrt(2.0 / math.pi) * 1.044715))
    np.testing.assert_allclose(oracle.activate(v, "gelu_tanh")[1:], [t - 1, 0, t, 30], rtol=1e-12)
    for kind in ("silu", "gelu", "gelu_tanh"):  # f(v) - f(-v) = v
        np.testing.assert_allclose(oracle.activate(v, kind) - oracle.activate(-v, kind), v, atol=1e-11)


def test_epilogue_pairs_the_halves():
    v = np.array([[1.0, -2.0, 3.0, 5.0]])
    r = np.array([[10.0, 20.0]])
    np.testing.assert_array_equal(oracle.epilogue(v, "relu", True, r), [[13.0, 20.0]])
    np.testing.assert_array_equal(oracle.epilogue(v, "relu", False), [[1.0, 0.0, 3.0, 5.0]])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_relative_angles(interleaved):
    rng = np.random.default_rng(1)
    hd, f = 16, 10000.0 ** (-np.arange(8) / 8)
    q, k = rng.standard_normal((2, 1, 1, hd))
    turn = lambda x, p: oracle.norm_rope(x, None, [p], f, eps=0.0, interleaved=interleaved)
    np.testing.assert_allclose(np.sum(turn(q, 12345) ** 2), np.sum(q ** 2), rtol=1e-12)
    dots = [np.sum(turn(q, 7 + p) * turn(k, 2 + p)) for p in (0, 1, 1000)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-9)
    # a quarter turn of one pair
    x = np.zeros((1, 1, 4))
    x[0, 0, 0] = 1.0
    y = oracle.norm_rope(x, None, [1], [math.pi / 2, 0.0], eps=0.0, interleaved=interleaved)
    want = np.zeros(4)
    want[1 if interleaved else 2] = 1.0
    np.testing.assert_allclose(y[0, 0], want, atol=1e-15)


def test_norm_of_each_head():
    x = np.array([[[3.0, 4.0], [0.0, 0.0]]])
    y = oracle.norm_rope(x, [1.0, 2.0], None, None, eps=0.5, interleaved=False)
    r = 1.0 / math.sqrt(13.0)
    np.testing.assert_allclose(y, [[[3 * r, 8 * r], [0.0, 0.0]]], rtol=1e-12)


def test_attention_by_hand():
    q = np.array([[0.0], [math.log(3.0)]])[:, None]     # two queries, one head
    k = np.array([[1.0], [0.0], [0.0]])[:, None]
    v = np.array([[1.0], [5.0], [9.0]])[:, None]
    cut = oracle.attention(q, k, v, [0, 2], [0], [3], scale=1.0, causal=True)
    np.testing.assert_allclose(cut[:, 0, 0], [3.0, (3 * 1 + 5 + 9) / 5.0], rtol=1e-12)
    # fewer keys than queries: the first query sees none
    short = oracle.attention(q, k, v, [0, 2], [2], [1], scale=1.0, causal=True)
    np.testing.assert_array_equal(short[:, 0, 0], [0.0, 9.0])
    none = oracle.attention(q, k, v, [0, 1], [0], [0], scale=1.0, causal=False)
    assert none[0, 0, 0] == 0.0 and np.isnan(none[1, 0, 0])


def test_attention_ignores_what_is_not_seen():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((3, 6, 2, 8))
    a = oracle.attention(q, k, v, [0, 6], [0], [6], scale=0.3, causal=True)
    k2, v2 = k.copy(), v.copy()
    k2[5], v2[5] = 100.0, 100.0
    b = oracle.attention(q, k2, v2, [0, 6], [0], [6], scale=0.3, causal=True)
    np.testing.assert_array_equal(a[:5], b[:5])
    assert np.all(a[5] != b[5])
    # one query at a time over the keys so far
    for i in range(6):
        one = oracle.attention(q[i:i + 1], k, v, [0, 1], [0], [i + 1], scale=0.3, causal=True)
        np.testing.assert_allclose(one[0], a[i], rtol=1e-12)
