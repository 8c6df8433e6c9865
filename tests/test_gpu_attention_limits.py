"""Attention at the ends of what a call may ask for: sequences of up to 2^31 - 1 keys."""
from __future__ import annotations

import pytest
import torch

from block_util import f64
from post_weight_quantization_syrk_amd import gptq
from serve_util import DEV, U16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    gptq.lib()


HD, ROWS, START = 8, 2 ** 31 + 100, 77


@pytest.fixture(scope="module")
def values():
    """Values of 2^31 keys (34 GB), all zero."""
    v = torch.zeros((ROWS, 1, HD), dtype=torch.bfloat16, device=DEV)
    yield v
    del v
    torch.cuda.empty_cache()


@pytest.mark.parametrize("tq", [1, 64])                      # few rows, and a tile of many
@pytest.mark.parametrize("lk", [2 ** 31 - 1, 2 ** 31 - 3000])
def test_every_key_of_the_longest_sequences_counts_once(values, tq, lk):
    """Scores are all 0, so a query's output is the mean of the values that it sees: one value of
    2^20 in each column, at keys where runs, tiles and 31 bits end, gives 2^20 over the keys seen.
    Weights are 1, their sums whole numbers that float32 has, so only the mean's rounding to bf16
    (half a step, 2^-8) and the quotient's (two of 2^-24) are off."""
    at = [0, 2 ** 24 + 5, 2 ** 30, 2080374784, 2 ** 31 - 65536, lk - tq - 200, lk - tq, lk - 1]
    values[START + torch.tensor(at, device=DEV), 0, torch.arange(HD, device=DEV)] = 2.0 ** 20
    zero = torch.zeros((1, 1, HD), dtype=torch.bfloat16, device=DEV)
    out = gptq.gptq_attention(zero.expand(tq, 1, HD), zero.expand(ROWS, 1, HD), values,
                              cu_q=torch.tensor([0, tq], dtype=torch.int32, device=DEV),
                              kv_start=torch.tensor([START], device=DEV),
                              kv_len=torch.tensor([lk], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    got = f64(out)[:, 0]
    values[START + torch.tensor(at, device=DEV)] = 0.0
    for i in range(tq):
        seen = lk - tq + 1 + i
        for c, j in enumerate(at):
            want = 2.0 ** 20 / seen if j < seen else 0.0
            assert abs(got[i, c] - want) <= (U16 + 2.0 ** -23) * want, (i, c, got[i, c], want)
