"""A prompt through the decoder block in one piece and in two, the second over the cache that the
first left: the same keys, values and attention, to the roundings that stand between."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from block_util import attention_reference, f64, linear_reference, rope_reference
from serve_util import DEV, U16
from test_gpu_decoder_block import EPS, HD, HK, HQ, D, State, block, i32, step  # noqa: F401

pytestmark = pytest.mark.gpu


def heads_bar(b, n1):
    """How far the block's queries, keys and values of one run may be from those of exact arithmetic
    on the same normalized rows: the product's bound e through the norm (y = x w r; r moves by at
    most sum |x| e / sum x^2 relative, twice that where e is not small beside x), the rotation (a
    pair's errors add) and the rounding to bf16, as the stages' own bars have it."""
    kw = b["qkv"]["kw"]
    v, e = linear_reference(f64(n1), *b["qkv"]["host"], kw["group_size"], kw["sym"], f64(b["bias"]), "none", False,
                            None, "f32")
    m = v.shape[0]
    x, e = v.reshape(m, HQ + 2 * HK, HD), e.reshape(m, HQ + 2 * HK, HD)
    pos, freq, half = np.arange(m), f64(b["freq"]), HD // 2
    out = []
    for lo, hi, w in ((0, HQ, f64(b["qn"])), (HQ, HQ + HK, f64(b["kn"]))):
        xs, es = x[:, lo:hi], e[:, lo:hi]
        y, own = rope_reference(xs, w, pos, freq, EPS, False)
        n = oracle.norm_rope(xs, w, None, None, eps=EPS, interleaved=False)
        r = 1.0 / np.sqrt(np.mean(xs * xs, axis=2, keepdims=True) + EPS)
        through = es * np.abs(w) * r + np.abs(n) * 2 * (np.abs(xs) * es).sum(2, keepdims=True) / (xs * xs).sum(2, keepdims=True)
        pair = through[:, :, :half] + through[:, :, half:]
        out.append((y, 1.01 * (own + np.concatenate([pair, pair], axis=2) * (1 + U16))))
    xs, es = x[:, HQ + HK:], e[:, HQ + HK:]
    out.append((xs, es + U16 * (np.abs(xs) + es)))
    return out


@pytest.mark.parametrize("n,cuts", [(133, [90]), (133, [1]), (133, [132]), (200, [64, 128]), (70, [30, 31, 69])])
def test_pieces_give_the_prompt(block, n, cuts):
    gen = torch.Generator(device=DEV).manual_seed(n + len(cuts))
    x = torch.randn((n, D), generator=gen, device=DEV).bfloat16()
    pos = torch.arange(n, device=DEV, dtype=torch.int32)
    runs = []
    for edges in ([0, n], [0, *cuts, n]):
        st = State()
        st.start, st.len = st.start[:1].clone(), st.len[:1].clone()
        n1, q, a = [], [], []
        for lo, hi in zip(edges, edges[1:]):
            st.len.fill_(hi)
            outs = step(block, x[lo:hi], st, pos[lo:hi].contiguous(), pos[lo:hi].long(), i32([0, hi - lo]))
            n1.append(outs[0]), q.append(outs[2]), a.append(outs[3])
        torch.cuda.synchronize()
        runs.append((torch.cat(n1), torch.cat(q), st.cache[0][:n].clone(), st.cache[1][:n].clone(), torch.cat(a)))
    assert torch.equal(runs[0][0], runs[1][0])        # a row's norm does not depend on the others
    # both runs' queries, keys and values against the same exact ones
    for i, (value, bar) in enumerate(heads_bar(block, runs[0][0])):
        for run in runs:
            assert np.all(np.abs(f64(run[1 + i]) - value) <= bar), i
    # outputs: each within its bar of exact attention on its own inputs, and these two apart by what
    # the inputs' differences d move: scores by scale (|dq||k| + |q||dk|), outputs by
    # sum w |ds| (|v| + |o|) + sum w |dv|, exponentials of ds at most 5% above 1 + ds here
    scale, group = HD ** -0.5, HQ // HK
    (_, q0, k0, v0, a0), (_, q1, k1, v1, a1) = [[f64(t) for t in run] for run in runs]
    o0, e0 = attention_reference(q0, k0, v0, [0, n], [0], [n], scale, True)
    o1, e1 = attention_reference(q1, k1, v1, [0, n], [0], [n], scale, True)
    for h in range(HQ):
        g = h // group
        w, _ = oracle.attention_weights(q0[:, h], k0[:, g], scale, True)
        ds = scale * (np.abs(q0[:, h] - q1[:, h]) @ np.maximum(np.abs(k0[:, g]), np.abs(k1[:, g])).T
                      + np.maximum(np.abs(q0[:, h]), np.abs(q1[:, h])) @ np.abs(k0[:, g] - k1[:, g]).T)
        assert (ds * (w > 0)).max() < 0.02
        moved = 1.05 * ((w * ds) @ np.abs(v0[:, g]) + (w * ds).sum(1, keepdims=True) * np.abs(o0[:, h])
                        + w @ np.abs(v0[:, g] - v1[:, g]))
        assert np.all(np.abs(a0[:, h] - a1[:, h]) <= e0[:, h] + e1[:, h] + moved), h
    assert float(np.abs(a0 - a1).max()) < 0.05 * float(np.abs(a0).max())
