"""What the bit-for-bit tests of the 4-bit products can see, on the CPU: a float32 sum in any order
gives the oracle's product exactly, and the oracle with a mistake planted in it does not."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from exact_util import exact_inputs


def product(x, words, s16, z16, g, sym):
    return oracle.dequant_matmul(x.astype(np.float64), words, s16, z16, bits=4, group_size=g, sym=sym)


@pytest.mark.parametrize("d_in,g,sym", [(2080, 32, False), (8192, 128, True), (65536, -1, False),
                                        (65536, 32, False)])
def test_sums_are_exact_in_float32(d_in, g, sym):
    x, _, words, s16, z16 = exact_inputs(2, d_in, 3, g, sym, d_in)
    ref = product(x, words, s16, z16, g, sym)
    W = oracle.dequantize(words, s16, z16, bits=4, group_size=g, sym=sym, d_in=d_in)
    rng = np.random.default_rng(1)
    for order in (np.arange(d_in), np.arange(d_in)[::-1], rng.permutation(d_in)):
        terms = (x[:, None, order] * W[None][:, :, order]).astype(np.float32)
        total = np.cumsum(terms, axis=2, dtype=np.float32)[:, :, -1]  # one after the other
        np.testing.assert_array_equal(total.astype(np.float64), ref)


@pytest.mark.parametrize("d_in,g", [(2080, 32), (8192, 128), (11008, 64), (32800, 32), (65536, -1)])
def test_planted_mistakes_show(d_in, g):
    m, d_out = 4, 64
    x, _, words, s16, z16 = exact_inputs(m, d_in, d_out, g, False, d_in + 1)
    ref = product(x, words, s16, z16, g, False)

    def share(wrong):
        return float((wrong != ref).mean())

    dropped = x.copy()
    dropped[:, -32:] = 0  # the last 32 k
    assert share(product(dropped, words, s16, z16, g, False)) > 0.9
    once_more = x.copy()
    once_more[:, :32] += x[:, d_in // 2:d_in // 2 + 32]  # 32 k against other weights as well
    assert share(product(once_more, words, s16, z16, g, False)) > 0.9
    swapped = x.reshape(m, -1, 2)[:, :, ::-1].reshape(m, d_in)  # even and odd codes
    assert share(product(swapped, words, s16, z16, g, False)) > 0.9
    if g != -1:  # a group's parameters taken from its neighbour
        assert share(product(x, words, np.roll(s16, 1, axis=1), z16, g, False)) > 0.9
        assert share(product(x, words, s16, np.roll(z16, 1, axis=1), g, False)) > 0.9
    assert share(product(x, words, s16, None, g, True)) > 0.5
