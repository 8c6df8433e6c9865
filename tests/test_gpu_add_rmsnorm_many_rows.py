"""GPU parity of gptq_add_rmsnorm past 1024 rows, where a row gets fewer threads with more
elements each, against the float64 oracle.  Bars as in test_gpu_add_rmsnorm.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from post_weight_quantization_syrk_amd import gptq
from test_gpu_add_rmsnorm import T, check, dev, out_buffer, untouched, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    gptq.lib()


# each width once in every pair of types; 8, 16 and 32 elements per thread, whole and ragged last
# pieces, a last wave with one thread's work, and the widths on either side of a step
TYPES = [("bf16", "bf16", "bf16"), ("f32", "bf16", "f32"), ("bf16", "f32", "bf16"),
         ("f32", "f32", "f32")]
WIDTHS = [520, 2047, 2048, 2049, 2056, 4096, 4097, 4104, 5003, 8184, 8192, 8193, 12288, 12289]


@pytest.mark.parametrize("ok", ["i8", "bf16"])
@pytest.mark.parametrize("i,d", list(enumerate(WIDTHS)))
@pytest.mark.parametrize("skewed", [False, True])
def test_add_rmsnorm_many_rows_match_oracle(i, d, skewed, ok):
    m = 1024 + 7 * i
    xk, rk, wk = TYPES[(i + skewed) % 4]
    pad, skew = (5, 1) if skewed else (0, 0)
    print(f"[norm] m={m} d={d} x={xk} r={rk} w={wk} out={ok} skewed={skewed}", flush=True)
    rng = np.random.default_rng([m, d])
    x, r, w = values(rng, m, d, xk, 0.3), values(rng, m, d, rk), values(rng, 1, d, wk)[0]
    X, R, W = dev(x, xk, pad, skew), dev(r, rk, pad, skew), dev(w[None], wk, 0, skew)[0]
    obuf, out = out_buffer(m, d, ok, pad, skew)
    rbuf, R_out = out_buffer(m, d, rk, pad, skew)
    o, s, h = gptq.gptq_add_rmsnorm(X, W, residual=R, residual_out=R_out, eps=1e-5,
                                    out_dtype=T[ok], out=out)
    torch.cuda.synchronize()
    check(x, r, w, rk, 1e-5, ok, o, s, h)
    assert untouched(obuf, out) and untouched(rbuf, R_out)
    # in place: the same bits
    o2, s2, h2 = gptq.gptq_add_rmsnorm(X, W, residual=R, residual_out=R, eps=1e-5,
                                       out_dtype=T[ok])
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(h, h2) and (s is None or torch.equal(s, s2))


@pytest.mark.parametrize("d", [2560, 2561, 5003, 8192])
def test_add_rmsnorm_either_side_of_1024_rows(d):
    """The same rows with 1023 others and with 1024: h and the codes are the same; the scale, whose
    sum is added in another order, within the two roundings of its bar."""
    rng = np.random.default_rng(d)
    x, r, w = values(rng, 1024, d, "bf16"), values(rng, 1024, d, "bf16"), values(rng, 1, d, "bf16")[0]
    X, R, W = dev(x, "bf16"), dev(r, "bf16"), dev(w[None], "bf16")[0]
    many = gptq.gptq_add_rmsnorm(X, W, residual=R, eps=1e-5)
    few = gptq.gptq_add_rmsnorm(X[:1023], W, residual=R[:1023], eps=1e-5)
    torch.cuda.synchronize()
    assert torch.equal(many[0][:1023], few[0]) and torch.equal(many[2][:1023], few[2])
    check(x, r, w, "bf16", 1e-5, "i8", *many)
    check(x[:1023], r[:1023], w, "bf16", 1e-5, "i8", *few)
