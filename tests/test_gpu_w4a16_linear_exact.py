"""The 4-bit product with its epilogue bit for bit, on inputs whose float32 sums are exact in any
order (exact_util): every form of tests/linear_forms.py, and rows of up to 65536 k, where the bar of
rounded sums is wider than a term that is left out.  The reference is the formula in float64 on the
GPU, itself compared with the oracle on some rows.  Gated outputs are the product of two exact sums,
rounded once."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from exact_util import exact_inputs
from linear_forms import FEW, TILES, WIDE
from post_weight_quantization_syrk_amd import gptq
from serve_util import DEV, dev_weights
from test_gpu_w4_exact import product

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    gptq.lib()


def compare(m, d_out, d_in, g, gated):
    sym = (m + d_out + d_in) % 2 == 0
    xi, _, words, s16, z16 = exact_inputs(m, d_in, d_out, g, sym, [m, d_in, d_out])
    Q, S, Z = dev_weights(words, s16, z16)
    X = torch.from_numpy(xi).to(DEV)
    ref = product(X.double(), Q, S, Z, d_in)
    some = np.unique(np.linspace(0, d_out - 1, 5).astype(int))
    np.testing.assert_array_equal(
        ref[:, some].cpu().numpy(),
        oracle.dequant_matmul(xi.astype(np.float64), words[some], s16[some], None if sym else z16[some], bits=4,
                              group_size=g, sym=sym))
    n = d_out
    if gated:
        n = d_out // 2
        ref = ref[:, :n] * ref[:, n:]
    room = torch.full((m * n + 64,), 77.0, dtype=torch.float32, device=DEV)
    Y = room[:m * n].view(m, n)
    gptq.gptq_w4a16_linear(X.bfloat16(), Q, S, Z, group_size=g, sym=sym, gated=bool(gated), out_dtype=torch.float32, Y=Y)
    torch.cuda.synchronize()
    assert bool((room[m * n:] == 77.0).all())
    wrong = (Y != ref.float()).nonzero()
    assert wrong.numel() == 0, f"{len(wrong)} of {Y.numel()} differ, first at {wrong[0].tolist()}"


@pytest.mark.parametrize("m,d_out,d_in,g,gated,form", FEW + TILES + WIDE)
def test_form(m, d_out, d_in, g, gated, form):
    compare(m, d_out, d_in, g, gated)


LONG = [(m, d_out, d_in, g, gated)
        for m, d_out in ((1, 34), (2, 66), (16, 50), (33, 34), (64, 18), (65, 66), (200, 130), (300, 514))
        for d_in, g in ((65536, 32), (65536, -1), (28704, 32), (65408, 64), (65408, 128)) for gated in (0, 1)]


@pytest.mark.parametrize("m,d_out,d_in,g,gated", LONG)
def test_long_rows(m, d_out, d_in, g, gated):
    compare(m, d_out, d_in, g, gated)
