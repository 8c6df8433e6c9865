"""GPU parity, bit for bit, of the two products with packed 4-bit weights (gptq_w4a16_matvec and
gptq_w4a8_matmul) on inputs whose float32 sums are exact in any order: over long rows, where the
bar of rounded sums says little, and over every launch shape of the one-token kernel (up to sixteen
waves to a row; 4, 8, 16 and 32 rows to a wave).

The reference is the formula in float64 on the GPU, itself compared with the oracle on some rows."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from exact_util import exact_inputs
from post_weight_quantization_syrk_amd import gptq
from serve_util import DEV, dev_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    gptq.lib()


def product(x64, Q, S, Z, d_in):
    """sum_k x (q - z) s in float64, some weight rows at a time."""
    d_out, ng = S.shape
    shifts = torch.arange(0, 32, 4, device=DEV, dtype=torch.int32)
    out = torch.empty((x64.shape[0], d_out), dtype=torch.float64, device=DEV)
    step = max(1, (1 << 26) // d_in)
    for n in range(0, d_out, step):
        q = ((Q[n:n + step, :, None] >> shifts) & 15).view(-1, ng, d_in // ng).double()
        q -= 8.0 if Z is None else Z[n:n + step].view(torch.float16).double()[:, :, None]
        q *= S[n:n + step].view(torch.float16).double()[:, :, None]
        out[:, n:n + step] = x64 @ q.view(-1, d_in).t().contiguous()
    return out


def compare(m, d_in, d_out, g, sym, i8):
    print(f"[exact] m={m} d_in={d_in} d_out={d_out} g={g} sym={sym} i8={i8}", flush=True)
    xi, xs, words, s16, z16 = exact_inputs(m, d_in, d_out, g, sym, [m, d_in, d_out])
    Q, S, Z = dev_weights(words, s16, z16)
    X = torch.from_numpy(xi).to(DEV)
    ref = product(X.double(), Q, S, Z, d_in)
    some = np.unique(np.linspace(0, d_out - 1, 5).astype(int))
    np.testing.assert_array_equal(
        ref[:, some].cpu().numpy(),
        oracle.dequant_matmul(xi.astype(np.float64), words[some], s16[some],
                              None if sym else z16[some], bits=4, group_size=g, sym=sym))
    Yg = torch.full((m * d_out + 64,), 77.0, dtype=torch.float32, device=DEV)
    Y = Yg[:m * d_out].view(m, d_out)
    if i8:
        XS = torch.from_numpy(xs).to(DEV)
        ref = ref * XS.double()[:, None]
        gptq.gptq_w4a8_matmul(X, XS, Q, S, Z, group_size=g, sym=sym, Y=Y)
    else:
        gptq.gptq_w4a16_matvec(X.bfloat16(), Q, S, Z, group_size=g, sym=sym, Y=Y)
    torch.cuda.synchronize()
    assert bool((Yg[m * d_out:] == 77.0).all())  # nothing behind the last row
    wrong = (Y.double() != ref).nonzero()
    assert wrong.numel() == 0, f"{len(wrong)} of {Y.numel()} differ, first at {wrong[0].tolist()}"


ONE_TOKEN = [
    # d_in, d_out, g, sym; 2048 k per wave
    (2048, 77, 64, False),
    (2080, 37, 32, False),       # a second wave with one lane's work
    (2080, 50, -1, True),
    (4128, 37, 32, True),        # three waves to a row
    (6176, 45, 32, False),       # four
    (6176, 45, -1, False),
    (8192, 300, 128, False),
    (11008, 131, 128, False),    # six
    (11008, 67, 64, True),
    (16416, 21, 32, False),      # nine
    (24608, 13, 32, False),      # thirteen
    (32768, 37, 128, False),     # sixteen: the longest row
    (32768, 9, -1, True),
    (32800, 37, 32, False),      # past it, the kernel for a few tokens
    (32800, 37, -1, False),
    (65536, 19, 64, False),
    (8192, 10003, 32, False),    # 8 rows per wave
    (32768, 2101, 128, False),   # 8, sixteen waves
    (28672, 2400, 64, True),     # 8, fourteen waves
    (8192, 28675, 128, False),   # 16
    (8192, 28675, -1, True),
    (2080, 40001, 32, False),    # 16, two waves
    (32768, 4200, -1, False),    # 16, sixteen waves
    (4096, 131075, 64, False),   # 32
    (32768, 8209, 64, False),    # 32, sixteen waves
    (1024, 130003, 128, True),   # 16, one wave to a row
    (1056, 262147, 32, False),   # 32
]


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("d_in,d_out,g,sym", ONE_TOKEN)
def test_one_token_is_exact(d_in, d_out, g, sym, i8):
    compare(1, d_in, d_out, g, sym, i8)


FEW_TOKENS = [
    # m, d_in, d_out, g, sym
    (2, 8192, 77, 128, False),
    (3, 11008, 4099, 32, False),
    (8, 65536, 19, 128, False),
    (16, 11008, 300, 64, True),
    (17, 32800, 40, 32, False),
    (32, 8192, 4100, -1, False),
    (33, 65536, 24, -1, False),
    (37, 11008, 4099, 32, False),
    (48, 32800, 35, -1, True),
    (49, 8160, 4100, 32, False),
    (64, 8192, 8190, 128, False),
    (64, 65536, 21, 64, False),
    (64, 11008, 6001, 64, True),
    (64, 32800, 70, 32, False),
]


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("m,d_in,d_out,g,sym", FEW_TOKENS)
def test_few_tokens_are_exact(m, d_in, d_out, g, sym, i8):
    compare(m, d_in, d_out, g, sym, i8)


@pytest.mark.parametrize("m,d_in,d_out,g,sym", [
    (65, 32800, 130, 32, False),
    (130, 8192, 300, 128, False),
    (200, 65536, 140, -1, False),
    (515, 11008, 1030, 64, True),
    (1000, 11008, 520, 32, False),
    (1500, 8192, 2050, 128, False),
    (2990, 8224, 2100, 32, False),
    (3030, 11040, 2090, -1, True),
    (160, 65536, 300, 64, False),
])
def test_many_tokens_are_exact(m, d_in, d_out, g, sym):
    compare(m, d_in, d_out, g, sym, True)
