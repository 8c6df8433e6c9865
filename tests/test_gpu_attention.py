"""GPU parity of attention over packed sequences and caches (gptq_attention) against the
float64 oracle; the bar is derived in block_util.attention_reference, before any run."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import oracle
from block_util import attention_reference, device, f64, randn, within
from post_weight_quantization_syrk_amd import gptq
from serve_util import DEV, replayed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    gptq.lib()


class Case:
    """lk None: packed keys; else each sequence's keys in a cache, its rows in no order."""

    def __init__(self, lq, lk, hq, hk, hd, causal=True, *, scale=None, before=0, behind=0, seed=0, hot=1.0):
        rng = np.random.default_rng([sum(lq), hq, hk, hd, seed])
        b = len(lq)
        self.causal, self.scale, self.hd = causal, scale, hd
        self.cu = np.concatenate([[before], before + np.cumsum(lq)]).astype(np.int64)
        tq = int(self.cu[-1]) + behind
        if lk is None:
            self.starts, self.lens, rows = self.cu[:-1], np.array(lq), tq
            self.start_d = self.len_d = None
        else:
            order = rng.permutation(b)
            self.starts, at = np.zeros(b, dtype=np.int64), 2
            for s in order:
                self.starts[s] = at
                at += lk[s] + int(rng.integers(0, 3))
            rows, self.lens = at + 1, np.array(lk)
            self.start_d = torch.from_numpy(self.starts).to(DEV)
            self.len_d = torch.from_numpy(self.lens.astype(np.int32)).to(DEV)
        self.q, self.q64 = device(hot * randn(rng, tq, hq, hd), "bf16")
        self.k, self.k64 = device(hot * randn(rng, rows, hk, hd), "bf16")
        self.v, self.v64 = device(randn(rng, rows, hk, hd), "bf16")
        self.cu_d = torch.from_numpy(self.cu.astype(np.int32)).to(DEV)

    def call(self, **kw):
        a = dict(cu_q=self.cu_d, kv_start=self.start_d, kv_len=self.len_d, causal=self.causal,
                 scale=self.scale) | kw
        q, k, v = (a.pop(n, getattr(self, n)) for n in ("q", "k", "v"))
        return gptq.gptq_attention(q, k, v, **a)

    def reference(self):
        scale = self.hd ** -0.5 if self.scale is None else self.scale
        return attention_reference(self.q64, self.k64, self.v64, self.cu, self.starts, self.lens, scale,
                                   self.causal)

    def check(self, out, what=""):
        y, e = self.reference()
        a, b = self.cu[0], self.cu[-1]
        within(out[a:b], y[a:b], e[a:b], what)


CASES = [
    # packed prompts: lengths of zero and one, odd ones, whole and ragged tiles, head sizes, groups
    dict(lq=[1], lk=None, hq=1, hk=1, hd=8),
    dict(lq=[0, 1, 0], lk=None, hq=2, hk=1, hd=16),
    dict(lq=[33], lk=None, hq=1, hk=1, hd=64, causal=False),
    dict(lq=[128], lk=None, hq=1, hk=1, hd=128),
    dict(lq=[129, 1, 200, 0, 63], lk=None, hq=4, hk=4, hd=128),
    dict(lq=[257, 300], lk=None, hq=8, hk=2, hd=64),
    dict(lq=[150, 77], lk=None, hq=5, hk=1, hd=80),
    dict(lq=[90, 210], lk=None, hq=6, hk=2, hd=96, causal=False),
    dict(lq=[100, 5], lk=None, hq=3, hk=1, hd=40),
    dict(lq=[190], lk=None, hq=2, hk=2, hd=136),
    dict(lq=[190], lk=None, hq=4, hk=2, hd=192, causal=False),
    dict(lq=[170, 31], lk=None, hq=4, hk=1, hd=256),
    dict(lq=[700], lk=None, hq=7, hk=7, hd=128),
    dict(lq=[40, 60], lk=None, hq=71, hk=1, hd=64),
    # pieces of prompts behind a cache; more queries than keys: rows that see nothing
    dict(lq=[64, 100], lk=[164, 100], hq=4, hk=2, hd=128),
    dict(lq=[130], lk=[1000], hq=8, hk=1, hd=128),
    dict(lq=[200, 50, 3], lk=[70, 0, 1], hq=2, hk=1, hd=64),
    dict(lq=[200, 50], lk=[1, 130], hq=2, hk=2, hd=128, causal=False),
    dict(lq=[300], lk=[299], hq=1, hk=1, hd=256),
    # next tokens over a cache: one to four to a sequence, keys over several workgroups
    dict(lq=[1], lk=[1], hq=8, hk=1, hd=128),
    dict(lq=[1], lk=[0], hq=8, hk=1, hd=128),
    dict(lq=[1], lk=[4096], hq=32, hk=8, hd=128),
    dict(lq=[1, 1, 1], lk=[31, 32, 33], hq=4, hk=4, hd=64),
    dict(lq=[1] * 9, lk=[0, 1, 63, 64, 65, 127, 128, 129, 1000], hq=8, hk=2, hd=128),
    dict(lq=[4, 2, 3], lk=[700, 2, 1], hq=8, hk=1, hd=128),
    dict(lq=[4, 4], lk=[515, 2], hq=5, hk=1, hd=80, causal=False),
    dict(lq=[2], lk=[3000], hq=2, hk=1, hd=256),
    dict(lq=[1, 1], lk=[900, 20], hq=16, hk=1, hd=192),
    dict(lq=[1] * 70, lk=[3 * i + 1 for i in range(70)], hq=2, hk=1, hd=64),
    dict(lq=[i % 3 for i in range(200)], lk=[i % 7 for i in range(200)], hq=1, hk=1, hd=32),
    dict(lq=[1] * 63 + [90], lk=[5] * 63 + [100], hq=2, hk=2, hd=96),
    dict(lq=[1], lk=[2500], hq=40, hk=1, hd=128),
    # scores far apart, another scale
    dict(lq=[150], lk=None, hq=2, hk=1, hd=128, hot=6.0),
    dict(lq=[1, 2], lk=[800, 300], hq=4, hk=1, hd=64, hot=6.0, scale=0.7),
    dict(lq=[65], lk=None, hq=2, hk=2, hd=64, scale=1e-6),
]


@pytest.mark.parametrize("kw", CASES, ids=lambda c: "-".join(str(v)[:40] for v in c.values()))
def test_attention(kw):
    c = Case(**kw)
    out = c.call()
    c.check(out)
    assert torch.equal(c.call(), out)  # the same bits again


@pytest.mark.parametrize("lq,lk", [([70, 40], None), ([1, 2], [300, 4])])
def test_rows_outside_all_sequences_stay(lq, lk):
    c = Case(lq, lk, 4, 2, 64, before=3, behind=9)
    out = torch.full_like(c.q, 7.0)
    c.call(out=out, max_kv_len=4096)
    c.check(out)
    assert bool((out[:3] == 7.0).all()) and bool((out[-9:] == 7.0).all())


@pytest.mark.parametrize("lq,lk", [([257], None), ([96, 140], [300, 150]), ([4, 3], [700, 90])])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), -3.3895e38, 3.3895e38])
def test_what_is_not_seen_does_not_matter(lq, lk, bad):
    """Causal: a key's and value's contents reach only the queries that see it; cache rows outside
    every sequence reach none."""
    c = Case(lq, lk, 4, 2, 128, seed=1)
    good = c.call()
    k, v = c.k.clone(), c.v.clone()
    used = np.zeros(k.shape[0], dtype=bool)
    for s, n in zip(c.starts, c.lens):
        used[s:s + n] = True
    outside = torch.from_numpy(np.nonzero(~used)[0]).to(DEV)
    k[outside], v[outside] = bad, bad
    assert torch.equal(c.call(k=k, v=v), good)
    # the third key from the end of each sequence: only its last three queries see it
    for s, n in zip(c.starts, c.lens):
        k[s + n - 3], v[s + n - 3] = bad, bad
    got = c.call(k=k, v=v)
    for i in range(len(lq)):
        a, b = c.cu[i], c.cu[i + 1]
        assert torch.equal(got[a:b - 3], good[a:b - 3]) or bool(torch.isfinite(got[a:b - 3]).all())
        y, e = c.reference()
        within(got[a:b - 3], y[a:b - 3], e[a:b - 3], f"sequence {i}")
        if not math.isfinite(bad):
            assert not bool(torch.isfinite(got[b - 3:b]).any())


@pytest.mark.parametrize("lq,lk", [([300, 40], None), ([3], [500]), ([140], [2000])])
@pytest.mark.parametrize("seen_too", [False, True])
def test_a_value_that_spoils_some_rows(lq, lk, seen_too):
    """A NaN in a value reaches the queries that see it, in its column and its heads alone, also
    where a value that they do not see is infinite."""
    c = Case(lq, lk, 4, 2, 96, seed=12)
    good = c.call()
    v = c.v.clone()
    n0, a0 = int(c.lens[0]), int(c.starts[0])
    first = n0 - lq[0] + 1                      # the second query sees it, the first does not
    v[a0 + first, 1, 7] = float("nan")
    if seen_too:
        v[a0 + n0 - 1, 1, 9] = float("inf")     # only the last query sees it
    got = c.call(v=v)
    a, b = int(c.cu[0]), int(c.cu[1])
    assert bool(torch.isnan(got[a + 1:b, 2:, 7]).all())
    y, e = c.reference()
    keep = [h for h in range(96) if h != 7]
    for rows, heads, cols in ((slice(a, a + 1), slice(0, 4), list(range(96))),
                              (slice(a + 1, b), slice(0, 2), list(range(96))),
                              (slice(a + 1, b - 1), slice(2, 4), keep)):
        within(got[rows, heads][:, :, cols], y[rows, heads][:, :, cols], e[rows, heads][:, :, cols])
    assert torch.equal(got[b:int(c.cu[-1])], good[b:int(c.cu[-1])])


@pytest.mark.parametrize("longest", [0, 1, 100, 100000])
def test_max_kv_len_is_only_a_hint(longest):
    for lq, lk in (([1, 1], [1500, 40]), ([150], [800])):
        c = Case(lq, lk, 8, 2, 128, seed=2)
        c.check(c.call(max_kv_len=longest), f"max {longest}")


def test_offsets_past_the_arrays_are_cut():
    c = Case([2, 2, 2, 2], [30, 30, 30, 30], 2, 1, 64, seed=3)
    rows = c.k.shape[0]
    start = torch.tensor([rows - 5, -7, rows + 100, 1 << 62], dtype=torch.int64, device=DEV)
    n = torch.tensor([50, 20, 3, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    got = c.call(kv_start=start, kv_len=n)
    c.starts, c.lens = np.array([rows - 5, 0, rows, rows]), np.array([5, 20, 0, 0])
    c.check(got)
    got = c.call(kv_start=start, kv_len=-n)
    assert bool((got == 0).all())
    # queries past the end, and a sequence that runs backwards
    cu = torch.tensor([0, 3, 2, 100, 1 << 30], dtype=torch.int32, device=DEV)
    assert c.call(cu_q=cu).shape == c.q.shape


def test_strides():
    """Heads outside rows, keys and values side by side, padded heads, shared (expanded) keys."""
    c = Case([90, 41], None, 4, 2, 64, seed=4)
    want = c.call()
    qt = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    kv = torch.zeros((131, 2, 2, 80), dtype=torch.bfloat16, device=DEV)
    kv[:, 0, :, :64], kv[:, 1, :, :64] = c.k, c.v
    out = torch.zeros((4, 131, 72), dtype=torch.bfloat16, device=DEV)[:, :, :64].transpose(0, 1)
    got = c.call(q=qt, k=kv[:, 0, :, :64], v=kv[:, 1, :, :64], out=out)
    assert torch.equal(got, want)
    a = c.call(k=c.k[:, :1].expand(131, 4, 64), v=c.v[:, :1].expand(131, 4, 64))
    b = c.call(k=c.k[:, :1], v=c.v[:, :1])
    within(a, f64(b), 2.0 ** -6 * np.abs(f64(b)) + 2.0 ** -7, "expanded")


def test_one_token_at_a_time_is_the_prompt():
    """The cache's form and the prompt's, on the same keys."""
    n, hq, hk, hd = 70, 4, 2, 128
    c = Case([n], None, hq, hk, hd, seed=5)
    whole = c.call()
    y, e = c.reference()
    for i in (0, 1, 31, 32, 63, 69):
        one = gptq.gptq_attention(c.q[i:i + 1], c.k, c.v,
                                  cu_q=torch.tensor([0, 1], dtype=torch.int32, device=DEV),
                                  kv_start=torch.zeros(1, dtype=torch.int64, device=DEV),
                                  kv_len=torch.tensor([i + 1], dtype=torch.int32, device=DEV))
        within(one[0], y[i], e[i], f"token {i}")
        within(whole[i], y[i], e[i], f"row {i}")


def test_nothing_to_do():
    q = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    cu = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert gptq.gptq_attention(q, q, q, cu_q=cu).shape == (0, 2, 64)
    q = torch.ones((3, 2, 64), dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, 7.0)
    gptq.gptq_attention(q, q, q, cu_q=cu, out=out)      # no sequence
    assert bool((out == 7.0).all())
    none = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    cu = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    gptq.gptq_attention(q, none, none, cu_q=cu, kv_start=zero, kv_len=zero.int() + 5, out=out)
    assert bool((out == 0).all())


@pytest.mark.parametrize("lq,lk", [([300], None), ([1, 1, 1], [2000, 5, 700])])
def test_captured_and_replayed(lq, lk):
    """Also with lengths that grow between the replays."""
    c = Case(lq, lk, 8, 2, 128, seed=6)
    want = c.call(max_kv_len=2000).cpu()
    out = torch.empty_like(c.q)
    ws = torch.empty(max(1, gptq.gptq_attention_workspace(c.q.shape[0], len(lq), 8, 2, 128, 2000)),
                     dtype=torch.uint8, device=DEV)
    longest = min(2000, c.k.shape[0])
    for (got,) in replayed(lambda: c.call(out=out, ws=ws, max_kv_len=longest), [out]):
        assert torch.equal(got, want) or c.check(got) is None
    if lk:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.call(out=out, ws=ws, max_kv_len=longest)
        for lens in ([1, 3, 2], [1900, 0, 650], [2000, 5, 700]):
            c.lens = np.array(lens)
            c.len_d.copy_(torch.tensor(lens, dtype=torch.int32))
            graph.replay()
            torch.cuda.synchronize()
            c.check(out, str(lens))


def test_two_calls_at_once():
    cs = [Case([1] * 3, [4000, 10, 900], 8, 1, 128, seed=7), Case([400], None, 8, 2, 64, seed=8)]
    want = [c.call() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        got = [c.call(stream=s) for c, s in zip(cs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_long_cache():
    """Keys and values past 2^31 elements, and rows that are 2^22 elements apart."""
    hd, rows = 128, (1 << 24) + 500
    K = torch.zeros((rows, 1, hd), dtype=torch.bfloat16, device=DEV)
    V = torch.zeros((rows, 1, hd), dtype=torch.bfloat16, device=DEV)
    c = Case([2, 70], [300, 200], 4, 1, hd, seed=9)
    at = [rows - 320, rows - 900]
    for s, (a, n) in enumerate(zip(at, (300, 200))):
        K[a:a + n] = c.k[c.starts[s]:c.starts[s] + n]
        V[a:a + n] = c.v[c.starts[s]:c.starts[s] + n]
    got = c.call(k=K, v=V, kv_start=torch.tensor(at, dtype=torch.int64, device=DEV), max_kv_len=300)
    c.check(got)
    wide = torch.zeros((520, 1, 1 << 22), dtype=torch.bfloat16, device=DEV)
    wide[:c.k.shape[0], :, :hd], wide[:c.k.shape[0], :, hd:2 * hd] = c.k, c.v
    got = c.call(k=wide[:c.k.shape[0], :, :hd], v=wide[:c.k.shape[0], :, hd:2 * hd])
    c.check(got)


@pytest.mark.parametrize("case", ["types", "heads", "V", "cu type", "cu shape", "len alone", "len type",
                                  "start shape", "packed rows", "out", "out type", "hd", "scale", "columns",
                                  "workspace", "unaligned", "overlap", "host"])
def test_refuses(case):
    c = Case([1, 1], [3000, 30], 4, 2, 64, seed=10)
    kw = {}
    if case == "types":
        kw["k"] = c.k.float()
    elif case == "heads":
        kw["q"] = c.q[:, :3]
    elif case == "V":
        kw["v"] = c.v[:-1]
    elif case == "cu type":
        kw["cu_q"] = c.cu_d.long()
    elif case == "cu shape":
        kw["cu_q"] = c.cu_d[None]
    elif case == "len alone":
        kw["kv_start"] = None
    elif case == "len type":
        kw["kv_len"] = c.len_d.long()
    elif case == "start shape":
        kw["kv_start"] = c.start_d[:1]
    elif case == "packed rows":
        kw.update(kv_start=None, kv_len=None)
    elif case == "out":
        kw["out"] = torch.zeros((2, 4, 63), dtype=torch.bfloat16, device=DEV)
    elif case == "out type":
        kw["out"] = torch.zeros((2, 4, 64), device=DEV)
    elif case == "hd":
        kw.update(q=c.q[:, :, :60], k=c.k[:, :, :60], v=c.v[:, :, :60])
    elif case == "scale":
        kw["scale"] = 0.0
    elif case == "columns":
        kw["q"] = c.q.transpose(1, 2).contiguous().transpose(1, 2)
    elif case == "workspace":
        kw["ws"] = torch.zeros(16, dtype=torch.uint8, device=DEV)
    elif case == "unaligned":
        kw["q"] = torch.zeros(2 * 4 * 64 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(2, 4, 64)
    elif case == "overlap":
        kw["out"] = torch.zeros((2, 64), dtype=torch.bfloat16, device=DEV)[:, None].expand(2, 4, 64)
    elif case == "host":
        kw["q"] = c.q.cpu()
    with pytest.raises((ValueError, gptq.GPTQError)):
        c.call(**kw)
