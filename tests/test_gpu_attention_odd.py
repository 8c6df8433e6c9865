"""Infinities and NaN in attention's keys and values: what a query sees of them gives what the
formula gives, in its column alone where they are values; what it does not see gives nothing.
The formula over the keys that a query sees, in float64 with IEEE arithmetic, is the reference;
finite outputs are held to block_util.attention_reference's bar on inputs whose odd values are 0."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_util import attention_reference, device, f64, randn
from post_weight_quantization_syrk_amd import gptq
from serve_util import DEV

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    gptq.lib()


class Case:
    """One sequence of lq queries over lk keys behind two rows of NaN."""

    def __init__(self, lq, lk, hq, hk, hd, causal, seed=0):
        rng = np.random.default_rng([lq, lk, hq, hk, hd, seed])
        self.lq, self.lk, self.hq, self.hk, self.hd, self.causal = lq, lk, hq, hk, hd, causal
        self.q, self.q64 = device(randn(rng, lq, hq, hd), "bf16")
        self.k, self.k64 = device(randn(rng, lk, hk, hd), "bf16")
        self.v, self.v64 = device(randn(rng, lk, hk, hd), "bf16")

    def put(self, t, at, value):
        """The value at the places (key, head, column) of keys or values."""
        for where in at:
            getattr(self, t)[where] = value
            getattr(self, t + "64")[where] = value

    def call(self, **kw):
        pad = torch.full((2, self.hk, self.hd), NAN, dtype=torch.bfloat16, device=DEV)
        k, v = torch.cat([pad, self.k, pad]), torch.cat([pad, self.v, pad])
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
        return gptq.gptq_attention(self.q, k, v, cu_q=i32([0, self.lq]), kv_len=i32([self.lk]), causal=self.causal,
                                   kv_start=torch.tensor([2], device=DEV), **kw)

    def seen(self, i):
        return max(0, self.lk - self.lq + 1 + i) if self.causal else self.lk

    def check(self, out, keys_as=None):
        """keys_as: float64 keys to take the finite outputs' bound with."""
        got, group, scale = f64(out), self.hq // self.hk, self.hd ** -0.5
        clean = np.where(np.isfinite(self.v64), self.v64, 0.0)
        _, bound = attention_reference(self.q64, self.k64 if keys_as is None else keys_as, clean, [0, self.lq], [0],
                                       [self.lk], scale, self.causal)
        odd = 0
        for i in range(self.lq):
            n = self.seen(i)
            for h in range(self.hq):
                k, v = self.k64[:n, h // group], self.v64[:n, h // group]
                if n == 0:
                    assert not got[i, h].any()
                    continue
                with np.errstate(invalid="ignore", over="ignore"):
                    s = (self.q64[i, h][None] * k).sum(1) * scale
                    w = np.exp(s - s.max())
                    want = (w[:, None] * v).sum(0) / w.sum()
                fin = np.isfinite(want)
                odd += int((~fin).sum())
                assert np.array_equal(np.isnan(got[i, h]), np.isnan(want)), (i, h)
                assert np.array_equal(got[i, h][np.isinf(want)], want[np.isinf(want)]), (i, h)
                err = np.abs(got[i, h][fin] - want[fin])
                assert np.all(err <= bound[i, h][fin]), (i, h, float((err / bound[i, h][fin]).max()))
        return odd


# few rows and many; ragged and whole tiles; keys over several workgroups
SHAPES = [(1, 1, 4, 1, 128), (1, 33, 4, 2, 64), (2, 64, 8, 1, 128), (1, 3000, 4, 1, 128), (3, 515, 2, 1, 80),
          (2, 700, 2, 1, 256), (40, 40, 2, 2, 128), (70, 133, 2, 1, 64), (65, 64, 4, 2, 96), (90, 1500, 2, 1, 128),
          (50, 301, 2, 1, 192), (45, 77, 2, 1, 256)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_the_last_value(shape, causal):
    """An infinity in the last key's value, whatever the number of keys leaves of a tile."""
    c = Case(*shape, causal)
    c.put("v", [(-1, 0, 0), (-1, 0, c.hd - 1)], INF)
    c.put("v", [(-1, c.hk - 1, 5)], -INF)
    assert c.check(c.call()) > 0


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_values_here_and_there(shape, causal):
    c = Case(*shape, causal, seed=1)
    n = c.lk
    c.put("v", [(0, 0, 1), (n // 2, 0, 1), (n // 3, 0, 7)], INF)
    c.put("v", [(n - 1, 0, 7), (n // 2, 0, 4)], -INF)          # column 7: both, where both are seen
    c.put("v", [(max(0, n - 2), 0, 2), (n // 2, c.hk - 1, 6)], NAN)
    assert c.check(c.call()) > 0


@pytest.mark.parametrize("lq,lk", [(1, 40), (1, 2500), (64, 64), (100, 900)])
def test_nothing_but_nan_behind_the_first_keys(lq, lk):
    """Causal rows in front of values that are all NaN keep theirs."""
    c = Case(lq, lk, 4, 2, 128, True, seed=2)
    at = max(1, lk - lq // 2)
    c.v[at:], c.v64[at:] = NAN, NAN
    c.check(c.call())
    if lq > 1:
        assert bool(torch.isfinite(c.call()[:lq // 2]).all())


@pytest.mark.parametrize("hd", [8, 24, 40, 72, 80, 104, 120, 136, 168, 200, 248])
@pytest.mark.parametrize("lq,lk", [(1, 50), (40, 100)])
def test_keys_whose_score_is_minus_infinity(lq, lk, hd):
    """An infinity in the last columns of a key, of the sign that makes its score -inf: the key has
    no weight, whether or not the head's columns fill whole blocks."""
    c = Case(lq, lk, 2, 1, hd, True, seed=3)
    c.q[:, :, hd - 1], c.q64[:, :, hd - 1] = 1.0, 1.0
    as_far = c.k64.copy()
    for j in (0, lk // 2, lk - 1):
        c.put("k", [(j, 0, hd - 1)], -INF)
        as_far[j, 0, hd - 1] = -100.0
    if lq == 1:
        # the only query; all of its keys but these three count
        assert bool(torch.isfinite(c.call()).all())
    c.check(c.call(), as_far)


@pytest.mark.parametrize("lq,lk,longest", [(1, 40, None), (1, 2000, None), (1, 700, 4096), (40, 70, None),
                                           (70, 1000, None)])
def test_no_finite_score(lq, lk, longest):
    """Rows that see keys whose scores are all -inf are 0 / 0; rows that see none stay 0."""
    c = Case(lq, lk, 2, 1, 64, True, seed=4)
    c.q[:, :, 3], c.q64[:, :, 3] = 1.0, 1.0
    c.k[:, :, 3], c.k64[:, :, 3] = -INF, -INF
    out = c.call(max_kv_len=longest)
    assert bool(torch.isnan(out[max(0, lq - lk):]).all())
    c = Case(lk, 3, 2, 1, 64, True, seed=5)     # most rows see none
    c.q[:, :, 3], c.k[:, :, 3] = 1.0, -INF
    out = c.call(max_kv_len=longest)
    assert bool((out[:-3] == 0).all()) and bool(torch.isnan(out[-3:]).all())


def test_a_prompt_of_nan_is_no_slower_by_orders():
    """4096 tokens whose values are NaN, against the same prompt clean: the rows are gone over again
    in tiles, some four times the work, not one by one (that took 400 times as long)."""
    n = 4096
    q, k, v = (torch.randn((n, h, 128), device=DEV).bfloat16() for h in (16, 4, 4))
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    least = []
    for bad in (False, True):
        if bad:
            v.fill_(NAN)
        times = []
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            out = gptq.gptq_attention(q, k, v, cu_q=cu)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        least.append(min(times))
    assert bool(torch.isnan(out).all())
    print(f"clean {least[0]:.3f} ms, NaN {least[1]:.3f} ms")
    assert least[1] < 30 * least[0]
