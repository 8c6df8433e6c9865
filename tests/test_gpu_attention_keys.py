"""Attention: every key counts once, and with few rows its weight has 17 bits.

On both paths (few rows: total_q times the heads of a key head up to 32 a sequence; many rows), in
one piece and with the keys split over workgroups."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import oracle
from block_util import device, f64, randn, within
from post_weight_quantization_syrk_amd import gptq
from serve_util import DEV, U16, U32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    gptq.lib()


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


# (queries, keys, query heads, key heads, hd, causal): tiles of 32 and 64 keys, waves' turns of 128,
# splits, heads of every width of the kernels
KEYS = [(1, 1, 1, 1, 64, True), (1, 33, 4, 1, 128, True), (1, 129, 8, 2, 96, True), (4, 300, 8, 1, 64, False),
        (1, 4096, 32, 8, 128, True), (3, 4099, 2, 1, 128, True), (1, 2300, 1, 1, 256, True), (2, 3001, 2, 1, 192, True),
        (33, 33, 1, 1, 64, True), (130, 130, 2, 1, 128, True), (64, 1000, 2, 1, 96, False), (100, 4100, 4, 1, 128, True),
        (256, 4096, 8, 2, 128, True), (70, 857, 2, 2, 256, True), (40, 1500, 1, 1, 192, True)]


@pytest.mark.parametrize("lq,lk,hq,hk,hd,causal", KEYS)
def test_every_key_counts_once(lq, lk, hq, hk, hd, causal):
    """Equal scores (queries of 0): a query's output is the mean of the values that it sees.  Each
    key in turn has the only value that is not 0 in its column; weights and their sums are whole
    numbers, so the mean is off by its quotient's and its own rounding alone.  A key left out gives
    0, one that counts twice, or for a query that does not see it, twice as much or not 0."""
    q = torch.zeros((lq, hq, hd), dtype=torch.bfloat16, device=DEV)
    k = torch.from_numpy(randn(np.random.default_rng(lk), lk, hk, hd)).to(DEV).bfloat16()
    seen = torch.arange(lq, device=DEV) + (lk - lq + 1) if causal else torch.full((lq,), lk, device=DEV)
    for first in range(0, lk, hd):
        v = torch.zeros((lk, hk, hd), dtype=torch.bfloat16, device=DEV)
        keys = torch.arange(first, min(lk, first + hd), device=DEV)
        v[keys, :, keys - first] = 1.0
        out = gptq.gptq_attention(q, k, v, cu_q=i32([0, lq]), kv_start=torch.zeros(1, dtype=torch.int64, device=DEV),
                                  kv_len=i32([lk]), causal=causal).double()
        want = torch.zeros((lq, hd), dtype=torch.float64, device=DEV)
        want[:, :len(keys)] = torch.where(keys[None] < seen[:, None], 1.0 / seen[:, None].double(), 0.0)
        err = (out - want[:, None]).abs()
        assert bool((err <= (U16 + 2 * U32) * want[:, None]).all()), (first, float(err.max()))


@pytest.mark.parametrize("lk,places", [(2, [0, 1]), (40, [0, 39]), (700, [3, 690]), (4096, [0, 4095]), (4096, [31, 32]),
                                       (4096, [1000, 3000])])
@pytest.mark.parametrize("hq,hk,hd", [(1, 1, 64), (4, 1, 128), (8, 2, 128), (2, 1, 256)])
def test_weights_of_few_rows_have_17_bits(lk, places, hq, hk, hd):
    """Two keys of scores d and 0 and values 1 and -1 give (1 - exp(-d)) over the sum of all weights:
    with weights of one bf16 part a d below 2^-9 would give 0.  The other keys' values are 0 and
    their scores 0 or, far below, weightless.

    Weights are off by 2^-17 relative (the first part leaves at most 2^-8 of the value's power of
    two, exactly, of which the second drops half a step, 2^-17), exp2 and its argument by 8 of 2^-24
    here (scores below 1), the sums by one rounding a key at most, of terms that are 0 but for two in
    the numerator."""
    rng = np.random.default_rng([lk, hd])
    d = np.exp2(rng.uniform(-12, -3, size=hq)).astype(np.float32)
    dq = torch.from_numpy(d).bfloat16()
    q = torch.zeros((1, hq, hd), dtype=torch.bfloat16, device=DEV)
    q[0, :, 0], q[0, :, 1] = dq.to(DEV), 1.0
    for rest in (0.0, -200.0):                # the other keys' scores
        k = torch.zeros((lk, hk, hd), dtype=torch.bfloat16, device=DEV)
        k[:, :, 1] = rest
        k[places[0], :, :2] = torch.tensor([1.0, 0.0], dtype=torch.bfloat16, device=DEV)
        k[places[1], :, :2] = 0.0
        v = torch.zeros((lk, hk, hd), dtype=torch.bfloat16, device=DEV)
        v[places[0]], v[places[1]] = 1.0, -1.0
        out = gptq.gptq_attention(q, k, v, cu_q=i32([0, 1]), kv_start=torch.zeros(1, dtype=torch.int64, device=DEV),
                                  kv_len=i32([lk]), scale=1.0)
        got = f64(out)[0]
        for h in range(hq):
            dd = float(dq[h])
            total = math.exp(dd) + 1.0 + (lk - 2) * math.exp(rest)
            want = (math.exp(dd) - 1.0) / total
            both = (math.exp(dd) + 1.0) / total
            e = (2.0 ** -17 + 12 * U32) * (both + abs(want)) + (lk + 64) * U32 * abs(want)
            assert np.all(np.abs(got[h] - want) <= e + U16 * (abs(want) + e)), (h, dd, want, got[h][:3], e)


def few_rows_reference(q, k, v, cu, starts, lens, scale):
    """block_util.attention_reference's value and bar for the path of few rows, whose weights are off
    by 2^-17 and not by half a step of bf16 (causal)."""
    tq, hq, hd = q.shape
    group = hq // k.shape[1]
    out, bound = np.zeros((tq, hq, hd)), np.zeros((tq, hq, hd))
    for s in range(len(cu) - 1):
        a, b, k0, n = cu[s], cu[s + 1], starts[s], lens[s]
        for h in range(hq):
            kk, vv = k[k0:k0 + n, h // group], v[k0:k0 + n, h // group]
            w, _ = oracle.attention_weights(q[a:b, h], kk, scale, True)
            o = w @ vv
            size = np.abs(q[a:b, h]) @ np.abs(kk).T * scale
            most = size.max(axis=1, initial=0.0)[:, None]
            delta = (hd + 8) * U32 * size + 8 * U32 * most + 4 * U32 + 2.0 ** -17 * (1 + 2.0 ** -7)
            e = (w * delta) @ np.abs(vv) + (w * delta).sum(1, keepdims=True) * np.abs(o)
            e += (2 * n + 64) * U32 * (w @ np.abs(vv) + np.abs(o))
            out[a:b, h], bound[a:b, h] = o, 1.05 * e + U16 * (np.abs(o) + e) + 1e-38
    return out, bound


@pytest.mark.parametrize("lq,lk,hq,hk,hd", [([1], [4096], 32, 8, 128), ([1] * 9, [1, 2, 31, 63, 64, 65, 129, 500, 1000], 8, 2, 128),
                                            ([4, 2, 3], [700, 2, 40], 8, 1, 128), ([2], [3000], 2, 1, 256),
                                            ([1, 1], [900, 20], 16, 1, 192), ([4, 4], [515, 9], 5, 1, 80),
                                            ([1] * 40, [37 * i + 1 for i in range(40)], 4, 2, 64)])
def test_few_rows_against_their_own_bar(lq, lk, hq, hk, hd):
    rng = np.random.default_rng([sum(lq), sum(lk), hd])
    cu, starts = np.concatenate([[0], np.cumsum(lq)]), np.concatenate([[0], np.cumsum(lk)[:-1]])
    assert sum(lq) * (hq // hk) <= 32 * len(lq)
    q, q64 = device(randn(rng, sum(lq), hq, hd), "bf16")
    k, k64 = device(randn(rng, sum(lk), hk, hd), "bf16")
    v, v64 = device(randn(rng, sum(lk), hk, hd), "bf16")
    for longest in (None, 1, max(lk)):
        out = gptq.gptq_attention(q, k, v, cu_q=i32(cu.tolist()), kv_start=torch.from_numpy(starts.astype(np.int64)).to(DEV),
                                  kv_len=i32(lk), max_kv_len=longest)
        within(out, *few_rows_reference(q64, k64, v64, cu, starts, lk, hd ** -0.5), f"longest {longest}")
