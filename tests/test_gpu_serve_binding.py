"""The binding's checks of shapes, types and devices for the calls that run a quantized
layer: each raises before the library is called, so nothing reaches the GPU."""
from __future__ import annotations

import pytest
import torch

from post_weight_quantization_syrk_amd import gptq
from serve_util import DEV

pytestmark = pytest.mark.gpu


def weights():
    return (torch.zeros((8, 32), dtype=torch.int32, device=DEV),
            torch.zeros((8, 2), dtype=torch.int16, device=DEV),
            torch.zeros((8, 2), dtype=torch.int16, device=DEV))


@pytest.mark.parametrize("case", ["qweight", "scales", "zeros", "missing zeros", "Y", "column-major",
                                  "3-D", "host scales", "float words"])
def test_products_refuse(case):
    Q, S, Z = weights()
    Y = None
    X = torch.zeros((2, 256), dtype=torch.bfloat16, device=DEV)
    if case == "qweight":
        Q = torch.zeros((8, 31), dtype=torch.int32, device=DEV)
    elif case == "scales":
        S = S[:, :1]
    elif case == "zeros":
        Z = Z[:4]
    elif case == "missing zeros":
        Z = None
    elif case == "Y":
        Y = torch.zeros((2, 9), device=DEV)
    elif case == "column-major":
        X = torch.zeros((256, 2), dtype=torch.bfloat16, device=DEV).t()
    elif case == "3-D":
        X = X[None]
    elif case == "host scales":
        S = S.cpu()
    elif case == "float words":
        Q = Q.float()
    with pytest.raises(ValueError):
        gptq.gptq_w4a16_matvec(X, Q, S, Z, group_size=128, sym=False, Y=Y)
    with pytest.raises(ValueError):
        gptq.gptq_w4a8_matmul(X.to(torch.int8), torch.zeros(2, device=DEV), Q, S, Z,
                              group_size=128, sym=False, Y=Y)


def test_products_refuse_through_the_library():
    Q, S, Z = weights()
    X = torch.zeros((2, 256), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(gptq.GPTQError) as e:
        gptq.gptq_w4a16_matvec(X, Q, S, Z, group_size=96, sym=False)
    assert e.value.status == gptq.GPTQ_EINVAL
    with pytest.raises(gptq.GPTQError) as e:
        gptq.gptq_w4a16_matvec(X[:1].expand(65, 256).contiguous(), Q, S, Z, group_size=128, sym=False)
    assert e.value.status == gptq.GPTQ_EUNSUPPORTED
    with pytest.raises(gptq.GPTQError) as e:  # rows that are one row
        gptq.gptq_w4a16_matvec(X[:1].expand(4, 256), Q, S, Z, group_size=128, sym=False)
    assert e.value.status == gptq.GPTQ_EINVAL
    with pytest.raises(ValueError):
        gptq.gptq_w4a8_matmul(X.to(torch.int8), torch.zeros(3, device=DEV), Q, S, Z,
                              group_size=128, sym=False)


@pytest.mark.parametrize("case", ["weight", "residual", "residual type", "sum without residual",
                                  "sum type", "out type", "out shape", "scales", "out_dtype",
                                  "column-major", "host residual"])
def test_add_rmsnorm_refuses(case):
    X = torch.zeros((2, 64), device=DEV)
    W = torch.ones(64, device=DEV)
    kw = dict(residual=torch.zeros((2, 64), device=DEV))
    if case == "weight":
        W = torch.ones(65, device=DEV)
    elif case == "residual":
        kw["residual"] = torch.zeros((2, 63), device=DEV)
    elif case == "residual type":
        kw["residual"] = torch.zeros((2, 64), dtype=torch.float16, device=DEV)
    elif case == "sum without residual":
        kw = dict(residual_out=torch.zeros((2, 64), device=DEV))
    elif case == "sum type":
        kw["residual_out"] = torch.zeros((2, 64), dtype=torch.bfloat16, device=DEV)
    elif case == "out type":
        kw["out"] = torch.zeros((2, 64), dtype=torch.bfloat16, device=DEV)
    elif case == "out shape":
        kw["out"] = torch.zeros((3, 64), dtype=torch.int8, device=DEV)
    elif case == "scales":
        kw["out_scales"] = torch.zeros(3, device=DEV)
    elif case == "out_dtype":
        kw["out_dtype"] = torch.float32
    elif case == "column-major":
        X = torch.zeros((64, 2), device=DEV).t()
    elif case == "host residual":
        kw["residual"] = torch.zeros((2, 64))
    with pytest.raises(ValueError):
        gptq.gptq_add_rmsnorm(X, W, **kw)
