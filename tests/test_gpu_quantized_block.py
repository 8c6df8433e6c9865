"""The layer-running calls together, as a quantized feed-forward block uses them, on weights
that the quantizer made: residual addition with the norm (8-bit output), the up projection in
8 bits, the down projection in bf16 for a few tokens, and the next norm, which takes the down
projection's fp32 output and updates the residual in place.

Each stage is held to its own bar on the inputs that it was given (the GPU's output of the
stage before), so no bar has to carry another stage's error."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from post_weight_quantization_syrk_amd import gptq
from serve_util import DEV, U16, U32, abs_terms

pytestmark = pytest.mark.gpu

D, F, EPS = 512, 1408, 1e-5


@pytest.fixture(scope="module")
def block():
    """Up [F, D] and down [D, F] projections, quantized from calibration activations."""
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    gen = torch.Generator(device=DEV).manual_seed(1)
    out = {"w_norm": (1 + 0.1 * torch.randn(D, generator=gen, device=DEV)).bfloat16()}
    for name, d_out, d_in, g, sym in (("up", F, D, 64, False), ("down", D, F, 128, True)):
        X = torch.randn((4 * d_in, d_in), generator=gen, device=DEV).bfloat16()
        H = torch.zeros((d_in, d_in), device=DEV)
        gptq.gptq_hessian_accumulate(H, X)
        U, dead, _ = gptq.gptq_prepare_hinv(H)
        W = 0.03 * torch.randn((d_out, d_in), generator=gen, device=DEV)
        codes, scales, zeros, _ = gptq.gptq_quantize_layer(W, U, dead, bits=4, group_size=g, sym=sym)
        q, s, z = gptq.gptq_pack(codes, scales, zeros, bits=4, group_size=g, sym=sym)
        torch.cuda.synchronize()
        host = (q.cpu().numpy().view(np.uint32), s.cpu().numpy().view(np.uint16),
                None if sym else z.cpu().numpy().view(np.uint16))
        out[name] = dict(dev=(q, s, z), host=host, g=g, sym=sym, d_in=d_in)
    return out


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def step(b, x, residual):
    """One block on x (the attention's output) and the residual, which is updated in place."""
    up, down = b["up"], b["down"]
    q8, qs, residual = gptq.gptq_add_rmsnorm(x, b["w_norm"], residual=residual,
                                             residual_out=residual, eps=EPS)
    h = gptq.gptq_w4a8_matmul(q8, qs, *up["dev"], group_size=up["g"], sym=up["sym"])
    a = torch.relu(h).bfloat16()
    call = gptq.gptq_w4a16_matvec if a.shape[0] <= gptq.GPTQ_MATVEC_MAX_M else gptq.gptq_w4a16_matmul
    y = call(a, *down["dev"], group_size=down["g"], sym=down["sym"])
    n, _, residual = gptq.gptq_add_rmsnorm(y, b["w_norm"], residual=residual, residual_out=residual,
                                           eps=EPS, out_dtype=torch.bfloat16)
    return q8, qs, h, a, y, n


@pytest.mark.parametrize("m", [1, 7, 64, 300])
def test_block(block, m):
    gen = torch.Generator(device=DEV).manual_seed(m)
    x = 0.3 * torch.randn((m, D), generator=gen, device=DEV)
    r = torch.randn((m, D), generator=gen, device=DEV).bfloat16()
    x0, r0 = x.cpu().numpy(), r.float().cpu().numpy()
    res = r.clone()
    q8, qs, h, a, y, n = step(block, x, res)
    torch.cuda.synchronize()
    w = f64(block["w_norm"])
    # first norm: codes exact, scales within half a step
    h0 = oracle.residual_sum(x0, r0, "bf16")
    codes, scale = oracle.norm_codes(h0, w, EPS)
    np.testing.assert_array_equal(q8.cpu().numpy(), codes)
    assert np.all(np.abs(f64(qs) - scale) <= U32 * (1 + 2.0 ** -10) * scale)
    # up projection on those codes
    up = block["up"]
    qw, s16, z16 = up["host"]
    What = oracle.dequantize(qw, s16, z16, bits=4, group_size=up["g"], sym=up["sym"], d_in=D)
    xq = codes.astype(np.float64) * f64(qs)[:, None]
    assert np.all(np.abs(f64(h) - xq @ What.T) <= (D / 32 + 4) * U32 * (np.abs(xq) @ np.abs(What).T))
    # down projection on the activations it was given
    down = block["down"]
    qw, s16, z16 = down["host"]
    ref = oracle.dequant_matmul(f64(a), qw, s16, z16, bits=4, group_size=down["g"], sym=down["sym"])
    bar = (F + 8) * U32 * (np.abs(f64(a)) @ abs_terms(qw, s16, z16, True, down["g"], F).T)
    assert np.all(np.abs(f64(y) - ref) <= bar)
    # second norm, and the residual after two additions in place
    h1 = oracle.residual_sum(y.cpu().numpy(), h0, "bf16")
    np.testing.assert_array_equal(res.float().cpu().numpy(), h1)
    ref = oracle.rms_norm(h1, w, EPS)
    assert np.all(np.abs(f64(n) - ref) <= (U16 + U32 + 2.0 ** -34) * np.abs(ref) + 2.0 ** -133)


@pytest.mark.parametrize("m", [1, 7, 300])
def test_block_captured_and_replayed(block, m):
    gen = torch.Generator(device=DEV).manual_seed(100 + m)
    x = 0.3 * torch.randn((m, D), generator=gen, device=DEV)
    r = torch.randn((m, D), generator=gen, device=DEV).bfloat16()
    res = r.clone()
    want = [t.clone() for t in step(block, x, res)]
    want_res = [res.clone()]
    for _ in range(2):  # the residual carries over from step to step
        again = step(block, x, res)
        want_res.append(res.clone())
    torch.cuda.synchronize()
    state = r.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(block, x, state)
    state.copy_(r)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(state, want_res[i])
        if i == 0:
            assert all(torch.equal(g, t) for g, t in zip(got, want))
        step(block, x, r.clone())  # eager work between the replays
    assert all(torch.equal(g, t) for g, t in zip(got, again))
