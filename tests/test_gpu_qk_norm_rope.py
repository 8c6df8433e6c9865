"""GPU parity of the norms of queries and keys with the rotation and the cache writes
(gptq_qk_norm_rope) against the float64 oracle; the bar is derived in
block_util.rope_reference, before any run."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_util import TORCH, device, f64, randn, rope_reference, within
from post_weight_quantization_syrk_amd import gptq
from serve_util import DEV, replayed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    gptq.lib()


class Case:
    def __init__(self, m, hq, hk, hd, rot, *, x="bf16", norm="bf16", pairs=False, first=0, seed=0,
                 eps=1e-6, with_v=True):
        rng = np.random.default_rng([m, hq, hk, hd, seed])
        heads = hq + 2 * hk
        self.m, self.hq, self.hk, self.hd, self.rot, self.eps, self.pairs = m, hq, hk, hd, rot, eps, pairs
        t, x64 = device(randn(rng, m, heads, hd) * np.exp(randn(rng, heads, 1)), x)
        self.q, self.k, self.v = t[:, :hq], t[:, hq:hq + hk], t[:, hq + hk:] if with_v else None
        self.x64 = (x64[:, :hq], x64[:, hq:hq + hk])
        self.qw = self.kw = self.qw64 = self.kw64 = None
        if norm:
            self.qw, self.qw64 = device(1 + 0.3 * randn(rng, hd), norm)
            self.kw, self.kw64 = device(1 + 0.3 * randn(rng, hd), norm)
        self.pos = (first + rng.integers(0, 4 * m + 1, size=m)).astype(np.int32)
        self.freq = None if rot == 0 else 500000.0 ** (-np.arange(0, rot, 2) / rot)
        self.pos_d = torch.from_numpy(self.pos).to(DEV)
        self.freq_d = None if rot == 0 else torch.from_numpy(self.freq).to(DEV)

    def call(self, **kw):
        a = dict(positions=self.pos_d, inv_freq=self.freq_d, q_weight=self.qw, k_weight=self.kw,
                 eps=self.eps, interleaved=self.pairs) | kw
        return gptq.gptq_qk_norm_rope(self.q, self.k, self.v, **a)

    def check(self, q, k, v):
        for name, got, x, w in (("q", q, self.x64[0], self.qw64), ("k", k, self.x64[1], self.kw64)):
            y, e = rope_reference(x, w, self.pos, self.freq, self.eps, self.pairs)
            within(got, y, e, name)
        if self.v is not None:
            assert torch.equal(v, self.v.to(torch.bfloat16))
        else:
            assert v is None


CASES = [
    dict(m=1, hq=1, hk=1, hd=8, rot=0),
    dict(m=1, hq=32, hk=8, hd=128, rot=128, x="f32"),
    dict(m=1, hq=32, hk=8, hd=128, rot=128, first=1 << 30),
    dict(m=2, hq=3, hk=1, hd=16, rot=16, norm=None, pairs=True),
    dict(m=3, hq=5, hk=5, hd=64, rot=64, norm="f32"),
    dict(m=5, hq=7, hk=2, hd=72, rot=32, x="f32", pairs=True),
    dict(m=7, hq=4, hk=4, hd=80, rot=80, first=1000000),
    dict(m=9, hq=4, hk=2, hd=80, rot=32, norm=None),
    dict(m=13, hq=6, hk=3, hd=96, rot=96, x="f32", norm="f32", pairs=True),
    dict(m=17, hq=2, hk=1, hd=256, rot=256),
    dict(m=19, hq=9, hk=1, hd=256, rot=64, pairs=True, first=-500),
    dict(m=33, hq=71, hk=1, hd=64, rot=48, x="f32"),
    dict(m=50, hq=16, hk=16, hd=120, rot=112, eps=0.1),
    dict(m=257, hq=8, hk=2, hd=128, rot=0, with_v=False),
    dict(m=1003, hq=21, hk=3, hd=80, rot=32, x="f32", norm=None, pairs=True),
    dict(m=3001, hq=8, hk=1, hd=128, rot=128),
    dict(m=9001, hq=2, hk=1, hd=64, rot=64, x="f32"),
    dict(m=9001, hq=2, hk=1, hd=40, rot=16, pairs=True, with_v=False),
]


@pytest.mark.parametrize("kw", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_rope(kw):
    c = Case(**kw)
    c.check(*c.call())


def test_only_one_norm():
    c = Case(6, 4, 2, 64, 64)
    q, k, _ = c.call(k_weight=None)
    within(q, *rope_reference(c.x64[0], c.qw64, c.pos, c.freq, c.eps, False), "q")
    within(k, *rope_reference(c.x64[1], None, c.pos, c.freq, c.eps, False), "k")


@pytest.mark.parametrize("m", [1, 37, 9000])
def test_slots(m):
    """Keys and values go to their rows; slots outside write nothing; other rows stay."""
    c = Case(m, 4, 2, 128, 128, seed=3)
    rows = 2 * m + 10
    rng = np.random.default_rng(m)
    slots = rng.permutation(rows)[:m].astype(np.int64)
    dense = c.call()
    for i, bad in enumerate((-1, rows, 1 << 40, -(1 << 62))):
        if m > 8 * i + 8:
            slots[8 * i + 1] = bad
    cache = torch.full((2, rows, 2, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    q, k, v = c.call(slots=torch.from_numpy(slots).to(DEV), k_out=cache[0], v_out=cache[1])
    assert torch.equal(q, dense[0])
    want = torch.full_like(cache, 5.0)
    ok = (slots >= 0) & (slots < rows)
    at, take = torch.from_numpy(slots[ok]).to(DEV), torch.from_numpy(np.nonzero(ok)[0]).to(DEV)
    want[0, at], want[1, at] = dense[1][take], dense[2][take]
    assert torch.equal(cache, want)


def test_the_same_slot_twice():
    """Each value is one of the two tokens'."""
    c = Case(2, 2, 1, 64, 64, seed=4)
    _, k, v = c.call()
    cache = torch.zeros((2, 3, 1, 64), dtype=torch.bfloat16, device=DEV)
    c.call(slots=torch.ones(2, dtype=torch.int64, device=DEV), k_out=cache[0], v_out=cache[1])
    for got, dense in zip(cache, (k, v)):
        assert bool(((got[1] == dense[0]) | (got[1] == dense[1])).all())
        assert bool((got[0] == 0).all() and (got[2] == 0).all())


def test_strides_and_in_place():
    """Heads outside tokens, padded rows, expanded inputs, outputs in the input's place."""
    c = Case(11, 4, 2, 64, 64, seed=5)
    want = c.call()
    q_out = torch.zeros((4, 11, 64), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    k_out = torch.zeros((11, 2, 72), dtype=torch.bfloat16, device=DEV)[:, :, :64]
    v_out = torch.zeros((11, 5, 64), dtype=torch.bfloat16, device=DEV)[:, 1:3]
    got = c.call(q_out=q_out, k_out=k_out, v_out=v_out)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    one = gptq.gptq_qk_norm_rope(c.q[:1, :1].expand(11, 4, 64), c.k, c.v, positions=c.pos_d,
                                 inv_freq=c.freq_d, q_weight=c.qw, k_weight=c.kw)[0]
    assert torch.equal(one[:, 0], one[:, 3])
    x = torch.cat([c.q, c.k, c.v], 1)
    got = gptq.gptq_qk_norm_rope(x[:, :4], x[:, 4:6], x[:, 6:], positions=c.pos_d, inv_freq=c.freq_d,
                                 q_weight=c.qw, k_weight=c.kw, q_out=x[:, :4], k_out=x[:, 4:6],
                                 v_out=x[:, 6:])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_far_positions():
    """Positions at the ends of int32, against the angle in float64."""
    c = Case(4, 2, 1, 128, 128, norm=None, x="f32", seed=6)
    c.pos = np.array([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 0], dtype=np.int32)
    c.pos_d = torch.from_numpy(c.pos).to(DEV)
    c.check(*c.call())


def test_empty_rows_and_zero_heads():
    c = Case(3, 2, 1, 64, 64, seed=7)
    e = gptq.gptq_qk_norm_rope(c.q[:0], c.k[:0], c.v[:0], positions=c.pos_d[:0], inv_freq=c.freq_d)
    assert [tuple(t.shape) for t in e] == [(0, 2, 64), (0, 1, 64), (0, 1, 64)]
    z = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device=DEV)
    q, k, _ = gptq.gptq_qk_norm_rope(z, z, positions=c.pos_d, inv_freq=c.freq_d, q_weight=c.qw,
                                     k_weight=c.kw)
    assert bool((q == 0).all()) and bool((k == 0).all())
    x = c.q.clone()
    x[1, 0, 5] = float("nan")   # one head's
    q, _, _ = gptq.gptq_qk_norm_rope(x, c.k, positions=c.pos_d, inv_freq=c.freq_d, q_weight=c.qw,
                                     k_weight=c.kw)
    good = c.call()[0]
    assert bool(torch.isnan(q[1, 0]).all())
    q[1, 0] = good[1, 0]
    assert torch.equal(q, good)


def test_no_tokens_leave_the_cache():
    c = Case(2, 2, 1, 64, 64, seed=11)
    cache = torch.full((2, 5, 1, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    e = gptq.gptq_qk_norm_rope(c.q[:0].clone(), c.k[:0].clone(), c.v[:0].clone(), positions=none.int(),
                               inv_freq=c.freq_d, slots=none, k_out=cache[0], v_out=cache[1])
    assert e[0].shape == (0, 2, 64) and bool((cache == 5.0).all())


@pytest.mark.parametrize("m", [1, 300])
def test_captured_and_replayed(m):
    c = Case(m, 8, 2, 128, 128, x="f32", seed=8)
    want = [t.cpu() for t in c.call()]
    outs = [torch.empty((m, h, 128), dtype=torch.bfloat16, device=DEV) for h in (8, 2, 2)]
    for got in replayed(lambda: c.call(q_out=outs[0], k_out=outs[1], v_out=outs[2]), outs):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_large_offsets():
    """A cache whose last rows lie past 2^31 elements."""
    c = Case(3, 2, 1, 64, 64, seed=9)
    rows, ld = 600, 1 << 22
    cache = torch.zeros((rows, ld), dtype=torch.bfloat16, device=DEV)
    k_out, v_out = cache[:, None, :64], cache[:, None, 64:128]
    slots = torch.tensor([599, 0, 598], dtype=torch.int64, device=DEV)
    c.call(slots=slots, k_out=k_out, v_out=v_out)
    _, k, v = c.call()
    assert torch.equal(k_out[slots], k) and torch.equal(v_out[slots], v)


@pytest.mark.parametrize("case", ["K heads", "V", "types", "positions", "positions type", "freq type",
                                  "no positions", "weight", "weight types", "slots type", "slots alone",
                                  "q_out", "k_out", "hd", "rot", "too much rot", "columns", "overlap",
                                  "unaligned", "v_out alone", "host"])
def test_refuses(case):
    c = Case(4, 4, 2, 64, 64, seed=10)
    q, k, v, kw = c.q, c.k, c.v, {}
    if case == "K heads":
        k = k[:, :, :32]
    elif case == "V":
        v = v[:, :1]
    elif case == "types":
        k = k.float()
    elif case == "positions":
        kw["positions"] = c.pos_d[:3]
    elif case == "positions type":
        kw["positions"] = c.pos_d.long()
    elif case == "freq type":
        kw["inv_freq"] = c.freq_d.float()
    elif case == "no positions":
        kw["positions"] = None
    elif case == "weight":
        kw["q_weight"] = c.qw[:32]
    elif case == "weight types":
        kw["q_weight"] = c.qw.float()
    elif case == "slots type":
        kw.update(slots=c.pos_d, k_out=k.clone(), v_out=v.clone())
    elif case == "slots alone":
        kw["slots"] = torch.arange(4, device=DEV)
    elif case == "q_out":
        kw["q_out"] = torch.zeros((4, 3, 64), dtype=torch.bfloat16, device=DEV)
    elif case == "k_out":
        kw["k_out"] = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device=DEV)
    elif case == "hd":
        q, k, v = (t[:, :, :60] for t in (q, k, v))
        kw.update(inv_freq=c.freq_d[:16], q_weight=None, k_weight=None)
    elif case == "rot":
        kw["inv_freq"] = c.freq_d[:12]
    elif case == "too much rot":
        kw["inv_freq"] = torch.ones(40, dtype=torch.float64, device=DEV)
    elif case == "columns":
        q = q.transpose(1, 2).contiguous().transpose(1, 2)
    elif case == "overlap":
        kw["q_out"] = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)[:, None].expand(4, 4, 64)
    elif case == "unaligned":
        q = torch.zeros(4 * 4 * 64 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(4, 4, 64)
    elif case == "v_out alone":
        v = None
        kw["v_out"] = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device=DEV)
    elif case == "host":
        q = q.cpu()
    a = dict(positions=c.pos_d, inv_freq=c.freq_d, q_weight=c.qw, k_weight=c.kw) | kw
    with pytest.raises((ValueError, gptq.GPTQError)):
        gptq.gptq_qk_norm_rope(q, k, v, **a)
