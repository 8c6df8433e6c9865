"""A whole quantized decoder block as a user runs it, on weights that the quantizer made: norm,
query/key/value product, norms of queries and keys with the rotation into a cache, attention,
output product onto the residual, norm, gate/up product, down product onto the residual.  First
prompts of different lengths, then tokens one by one, eager and captured.

Each stage is held to its own bar on the inputs that it was given (the GPU's output of the
stage before), so no bar has to carry another stage's error."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from block_util import attention_reference, f64, linear_reference, rope_reference, within
from post_weight_quantization_syrk_amd import gptq
from serve_util import DEV, U16, U32

pytestmark = pytest.mark.gpu

D, F, HQ, HK, HD, EPS = 512, 768, 8, 2, 64, 1e-5
CAP = 400                       # cache rows per sequence
PROMPTS = [70, 1, 133]


@pytest.fixture(scope="module")
def block():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    gen = torch.Generator(device=DEV).manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=gen, device=DEV)
    b = {n: (1 + 0.1 * rand(k)).bfloat16() for n, k in (("n1", D), ("n2", D), ("qn", HD), ("kn", HD))}
    b["freq"] = 10000.0 ** (-torch.arange(0, HD, 2, device=DEV, dtype=torch.float64) / HD)
    b["bias"] = (0.1 * rand((HQ + 2 * HK) * HD)).bfloat16()
    for name, outs, d_in, g, sym in (("qkv", [HQ * HD, HK * HD, HK * HD], D, 64, False),
                                     ("o", [D], HQ * HD, 128, True), ("gu", [F, F], D, 32, False),
                                     ("down", [D], F, 64, False)):
        X = rand(4 * d_in, d_in).bfloat16()
        H = torch.zeros((d_in, d_in), device=DEV)
        gptq.gptq_hessian_accumulate(H, X)
        U, dead, _ = gptq.gptq_prepare_hinv(H)
        Ws = [0.04 * rand(n, d_in) for n in outs]
        codes, scales, zeros = gptq.gptq_quantize_layers(Ws, U, dead, bits=4, group_size=g, sym=sym)[:3]
        q, s, z = gptq.gptq_pack(codes, scales, zeros, bits=4, group_size=g, sym=sym)
        torch.cuda.synchronize()
        b[name] = dict(w=(q, s, z), kw=dict(group_size=g, sym=sym),
                       host=(q.cpu().numpy().view(np.uint32), s.cpu().numpy().view(np.uint16),
                             None if sym else z.cpu().numpy().view(np.uint16)))
    return b


def linear(b, name, x, **kw):
    return gptq.gptq_w4a16_linear(x, *b[name]["w"], **b[name]["kw"], **kw)


class State:
    def __init__(self):
        self.cache = torch.zeros((2, len(PROMPTS) * CAP, HK, HD), dtype=torch.bfloat16, device=DEV)
        self.start = torch.arange(len(PROMPTS), device=DEV) * CAP
        self.len = torch.zeros(len(PROMPTS), dtype=torch.int32, device=DEV)


def step(b, x, st, pos, slots, cu):
    """One block on the residual stream x [m, D] bf16; returns every stage's output."""
    m = x.shape[0]
    n1 = gptq.gptq_add_rmsnorm(x, b["n1"], eps=EPS, out_dtype=torch.bfloat16)[0]
    qkv = linear(b, "qkv", n1, bias=b["bias"], out_dtype=torch.float32).view(m, HQ + 2 * HK, HD)
    q, _, _ = gptq.gptq_qk_norm_rope(qkv[:, :HQ], qkv[:, HQ:HQ + HK], qkv[:, HQ + HK:], positions=pos,
                                     inv_freq=b["freq"], q_weight=b["qn"], k_weight=b["kn"], eps=EPS,
                                     slots=slots, k_out=st.cache[0], v_out=st.cache[1])
    a = gptq.gptq_attention(q, st.cache[0], st.cache[1], cu_q=cu, kv_start=st.start, kv_len=st.len,
                            max_kv_len=CAP)
    x1 = linear(b, "o", a.view(m, HQ * HD), residual=x, Y=x.clone())
    n2 = gptq.gptq_add_rmsnorm(x1, b["n2"], eps=EPS, out_dtype=torch.bfloat16)[0]
    h = linear(b, "gu", n2, activation="silu", gated=True)
    y = linear(b, "down", h, residual=x1)
    return n1, qkv, q, a, x1, n2, h, y


def check(b, x, st, pos, slots, cu, outs):
    n1, qkv, q, a, x1, n2, h, y = outs
    P, S = pos.cpu().numpy(), slots.cpu().numpy()

    def product(name, x, got, what, bias=None, act="none", gated=False, res=None, out="bf16"):
        kw = b[name]["kw"]
        v, e = linear_reference(f64(x), *b[name]["host"], kw["group_size"], kw["sym"], bias, act, gated, res, out)
        within(got, v, e, what)

    norm = lambda x, w: oracle.rms_norm(f64(x), f64(w), EPS)
    for got, src, w in ((n1, x, b["n1"]), (n2, x1, b["n2"])):
        v = norm(src, w)
        assert np.all(np.abs(f64(got) - v) <= (U16 + D * U32) * np.abs(v) + 1e-38)
    product("qkv", n1, qkv.reshape(len(P), -1), "qkv", bias=f64(b["bias"]), out="f32")
    q64 = f64(qkv)
    within(q, *rope_reference(q64[:, :HQ], f64(b["qn"]), P, f64(b["freq"]), EPS, False), "queries")
    within(st.cache[0][slots], *rope_reference(q64[:, HQ:HQ + HK], f64(b["kn"]), P, f64(b["freq"]), EPS, False),
           "keys")
    assert torch.equal(st.cache[1][slots], qkv[:, HQ + HK:].bfloat16())
    within(a, *attention_reference(f64(q), f64(st.cache[0]), f64(st.cache[1]), cu.cpu().numpy(),
                                   st.start.cpu().numpy(), st.len.cpu().numpy(), HD ** -0.5, True), "attention")
    product("o", a.reshape(len(P), -1), x1, "out", res=f64(x))
    product("gu", n2, h, "gate/up", act="silu", gated=True)
    product("down", h, y, "down", res=f64(x1))


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def test_prompts_then_tokens(block):
    gen = torch.Generator(device=DEV).manual_seed(2)
    st = State()
    x = torch.randn((sum(PROMPTS), D), generator=gen, device=DEV).bfloat16()
    pos = torch.cat([torch.arange(n, device=DEV, dtype=torch.int32) for n in PROMPTS])
    slots = torch.cat([s * CAP + torch.arange(n, device=DEV) for s, n in enumerate(PROMPTS)])
    st.len.copy_(i32(PROMPTS))
    cu = i32([0, *np.cumsum(PROMPTS)])
    outs = step(block, x, st, pos, slots, cu)
    torch.cuda.synchronize()
    check(block, x, st, pos, slots, cu, outs)
    # tokens one by one: one captured step, its lengths, positions and slots moved on before each replay
    b = len(PROMPTS)
    tx = torch.randn((b, D), generator=gen, device=DEV).bfloat16()
    tpos, tslots, tcu = i32(PROMPTS), torch.tensor([s * CAP + n for s, n in enumerate(PROMPTS)], device=DEV), i32(range(b + 1))
    st.len.copy_(i32([n + 1 for n in PROMPTS]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(block, tx, st, tpos, tslots, tcu)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        touts = step(block, tx, st, tpos, tslots, tcu)
    for t in range(4):
        tx.copy_(torch.randn((b, D), generator=gen, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        check(block, tx, st, tpos, tslots, tcu, touts)
        eager = step(block, tx, st, tpos, tslots, tcu)
        assert all(torch.equal(p, q) for p, q in zip(eager, touts))
        tpos += 1
        tslots += 1
        st.len += 1


def test_prompt_in_pieces_is_the_prompt(block):
    """A prompt in two pieces, the second over the cache the first left: the same stream, to the
    roundings of the weights that stand between."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    n, cut = 133, 90
    x = torch.randn((n, D), generator=gen, device=DEV).bfloat16()
    pos = torch.arange(n, device=DEV, dtype=torch.int32)
    ys = []
    for pieces in ([(0, n)], [(0, cut), (cut, n)]):
        st = State()
        st.start, st.len = st.start[:1].clone(), st.len[:1].clone()
        got = []
        for a, z in pieces:
            st.len.fill_(z)
            outs = step(block, x[a:z], st, pos[a:z].contiguous(), pos[a:z].long(), i32([0, z - a]))
            got.append(outs[3])
            check(block, x[a:z], st, pos[a:z], pos[a:z].long(), i32([0, z - a]), outs)
        ys.append(torch.cat(got))
    assert ys[0].shape == ys[1].shape
