"""Inputs for which the 4-bit products are exact in float32, whatever the order of the sums
(no step of the method here).

x is a whole number of -2 .. 2, zeros are whole numbers of 0 .. 15, and scales 2^-6 .. 2^-3.
A group's sums of x q and z sum x are whole numbers of at most 2 15 K; the total, in units of
2^-6, is at most 2 15 8 K.  For K <= 65536 every partial sum is thus a whole number of such
units below 2^24: each addition is exact, and a term left out, taken twice or multiplied by
another group's parameters shows in the last bit."""
from __future__ import annotations

import numpy as np

assert 2 * 15 * 8 * 65536 < 2 ** 24


def exact_inputs(m, d_in, d_out, g, sym, seed):
    """(x int8 [m, d_in], x_scales float32 [m], words uint32, scales bits, zeros bits or None)."""
    rng = np.random.default_rng(seed)
    ng = 1 if g == -1 else d_in // g
    x = rng.integers(-2, 3, size=(m, d_in), dtype=np.int8)
    xs = np.exp2(rng.integers(-4, 4, size=m)).astype(np.float32)
    words = rng.integers(0, 2 ** 32, size=(d_out, d_in // 8), dtype=np.uint32)
    s16 = np.exp2(rng.integers(-6, -2, size=(d_out, ng))).astype(np.float16).view(np.uint16)
    z16 = rng.integers(0, 16, size=(d_out, ng)).astype(np.float16).view(np.uint16)
    return x, xs, words, s16, None if sym else z16
