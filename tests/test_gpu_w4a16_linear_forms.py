"""Every form of the 4-bit product with its epilogue (tests/linear_forms.py: tiles of tokens and
weight rows, waves that share the tokens, splits, blocks of rows, weights in eight bits) against the
float64 oracle, inside block_util.linear_reference's bound."""
from __future__ import annotations

import pytest
import torch

from linear_forms import FEW, TILES, WIDE
from post_weight_quantization_syrk_amd import gptq
from test_gpu_w4a16_linear import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    gptq.lib()


@pytest.mark.parametrize("m,d_out,d_in,g,gated,form", FEW + TILES + WIDE)
def test_form(m, d_out, d_in, g, gated, form):
    i = m + d_out + d_in + g
    c = Case(m, d_in, d_out, g, bool(i % 2), gated=bool(gated), act=("silu" if gated else ("none", "relu", "silu")[i % 3]),
             bias=(None, "bf16", "f32")[i % 3], res=(None, "f32", "bf16")[i // 2 % 3], out=("f32", "bf16")[i // 3 % 2],
             pad=i % 2)
    Y = c.call()
    c.check(Y, form)
    assert torch.equal(c.call(), Y)


@pytest.mark.parametrize("m,d_out,d_in,g,gated,form", [c for c in WIDE if c[0] == 1355])
def test_eight_bit_weights_captured(m, d_out, d_in, g, gated, form):
    """The weights are made wide in the graph too: other weights give other outputs."""
    c = Case(m, d_in, d_out, g, False, gated=bool(gated), act="silu")
    d = Case(m, d_in, d_out, g, False, gated=bool(gated), act="silu", seed=1)
    d.X.copy_(c.X)
    want = c.call(), d.call()
    Y = torch.empty_like(want[0])
    ws = torch.empty(gptq.gptq_w4a16_linear_workspace(m, d_out, d_in, g, bool(gated)), dtype=torch.uint8, device=Y.device)
    weights = [t.clone() for t in c.dev]
    call = lambda: gptq.gptq_w4a16_linear(c.X, *weights, group_size=g, sym=False, gated=bool(gated), activation="silu",
                                          Y=Y, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in (1, 0, 1):
        for t, s in zip(weights, (c, d)[k].dev):
            t.copy_(s)
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want[k])
