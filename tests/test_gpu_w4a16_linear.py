"""GPU parity of the 4-bit product with bias, activation, gate and residual
(gptq_w4a16_linear) against the float64 oracle; the bar is derived in
block_util.linear_reference, before any run."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_util import TORCH, device, f64, linear_reference, padded, randn, weights, within
from post_weight_quantization_syrk_amd import gptq, synth
from serve_util import DEV, dev_weights, replayed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    gptq.lib()


class Case:
    def __init__(self, m, d_in, d_out, g, sym, *, bias=None, act="none", gated=False, res=None,
                 out="bf16", pad=0, seed=0):
        rng = np.random.default_rng([m, d_in, d_out, seed])
        self.g, self.sym, self.act, self.gated, self.out = g, sym, act, gated, out
        self.m, self.n = m, d_out // 2 if gated else d_out
        self.packed = weights(d_in, d_out, g, sym, seed + 7)
        x = randn(rng, m, d_in) * np.exp(0.5 * randn(rng, d_in)) / np.sqrt(d_in)
        X, self.x64 = device(x, "bf16")
        self.X = padded(X, 8 * pad)
        self.bias, self.b64 = device(randn(rng, d_out), bias) if bias else (None, None)
        self.res = self.r64 = None
        if res:
            r, self.r64 = device(2 * randn(rng, m, self.n), res)
            self.res = padded(r, pad)
        self.dev = dev_weights(*self.packed)

    def call(self, **kw):
        a = dict(group_size=self.g, sym=self.sym, bias=self.bias, activation=self.act,
                 gated=self.gated, residual=self.res, out_dtype=TORCH[self.out]) | kw
        return gptq.gptq_w4a16_linear(self.X, *self.dev, **a)

    def check(self, Y, what=""):
        y, e = linear_reference(self.x64, *self.packed, self.g, self.sym, self.b64, self.act,
                                self.gated, self.r64, self.out)
        assert Y.dtype == TORCH[self.out]
        within(Y, y, e, what)


CASES = [
    # few tokens: one token, 2 to 64, splits, shared buffers
    dict(m=1, d_in=32, d_out=1, g=32, sym=False, bias="f32", act="relu"),
    dict(m=1, d_in=64, d_out=2, g=64, sym=True, gated=True, act="silu"),
    dict(m=1, d_in=256, d_out=33, g=128, sym=False, bias="bf16", res="bf16", act="gelu"),
    dict(m=1, d_in=4096, d_out=514, g=64, sym=False, gated=True, act="gelu_tanh", bias="f32", res="f32", out="f32"),
    dict(m=1, d_in=65536, d_out=6, g=32, sym=False, gated=True, act="silu", bias="bf16"),
    dict(m=1, d_in=1056, d_out=70, g=-1, sym=True, act="silu", out="f32", pad=3),
    dict(m=2, d_in=96, d_out=62, g=32, sym=False, gated=True, act="relu", res="bf16", pad=1),
    dict(m=3, d_in=1056, d_out=100, g=32, sym=True, act="gelu", bias="f32", pad=1),
    dict(m=5, d_in=544, d_out=130, g=-1, sym=False, gated=True, act="silu", res="f32", out="f32", pad=5),
    dict(m=16, d_in=4096, d_out=200, g=128, sym=False, act="silu", bias="bf16", res="f32"),
    dict(m=16, d_in=640, d_out=9000, g=64, sym=True, gated=True, act="silu"),
    dict(m=17, d_in=2208, d_out=48, g=32, sym=False, gated=True, act="gelu_tanh", bias="f32"),
    dict(m=33, d_in=4096, d_out=66, g=64, sym=False, act="none", res="bf16", bias="bf16"),
    dict(m=40, d_in=6272, d_out=300, g=128, sym=False, gated=True, act="silu", res="bf16"),
    dict(m=49, d_in=4160, d_out=12290, g=64, sym=False, gated=True, act="gelu", bias="bf16"),
    dict(m=64, d_in=6176, d_out=8190, g=-1, sym=False, act="relu", res="f32", out="f32"),
    dict(m=64, d_in=5152, d_out=2102, g=-1, sym=False, gated=True, act="silu", bias="f32"),
    # few tokens through large weights
    dict(m=50, d_in=1056, d_out=25801, g=32, sym=False, act="silu", bias="bf16", res="f32"),
    dict(m=57, d_in=4160, d_out=10880, g=64, sym=True, gated=True, act="gelu", out="f32"),
    # tiles: ragged rows, columns and k, splits, every group size
    dict(m=65, d_in=32, d_out=1, g=32, sym=False, act="relu", bias="f32", res="bf16"),
    dict(m=65, d_in=96, d_out=2, g=32, sym=True, gated=True, act="silu"),
    dict(m=70, d_in=160, d_out=129, g=-1, sym=False, act="gelu", out="f32", pad=1),
    dict(m=97, d_in=1088, d_out=131, g=64, sym=False, act="gelu_tanh", res="f32", pad=3),
    dict(m=100, d_in=4128, d_out=67, g=32, sym=False, bias="bf16", out="f32"),
    dict(m=128, d_in=2048, d_out=520, g=128, sym=False, gated=True, act="silu", res="bf16", bias="f32", pad=4),
    dict(m=130, d_in=4096, d_out=4100, g=64, sym=True, act="silu", bias="bf16"),
    dict(m=200, d_in=11008, d_out=190, g=128, sym=False, act="none", res="bf16"),
    dict(m=257, d_in=480, d_out=514, g=32, sym=False, gated=True, act="relu", out="f32"),
    dict(m=515, d_in=736, d_out=1027, g=32, sym=False, act="gelu", res="f32", out="f32"),
    dict(m=600, d_in=672, d_out=7000, g=-1, sym=False, gated=True, act="silu"),
    dict(m=1000, d_in=256, d_out=8193, g=128, sym=True, act="none", bias="f32"),
    dict(m=2049, d_in=192, d_out=4224, g=64, sym=False, gated=True, act="gelu_tanh", res="bf16"),
    dict(m=2100, d_in=320, d_out=5000, g=32, sym=True, act="silu", out="f32"),
    dict(m=3000, d_in=128, d_out=3001, g=128, sym=False, act="relu", res="bf16", pad=7),
]


@pytest.mark.parametrize("kw", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_linear(kw):
    c = Case(**kw)
    Y = c.call()
    c.check(Y)
    # into rows that are longer, what lies behind them untouched; twice the same bits
    wide = torch.full((c.m, c.n + 5), 7.0, dtype=Y.dtype, device=DEV)
    got = c.call(Y=wide[:, :c.n])
    assert torch.equal(got, Y) and bool((wide[:, c.n:] == 7.0).all())


@pytest.mark.parametrize("m", [1, 20, 300])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("gated", [False, True])
def test_residual_in_place(m, kind, gated):
    c = Case(m, 512, 260, 128, False, act="silu", gated=gated, res=kind, out=kind)
    want = c.call()
    r = c.res.clone()
    got = gptq.gptq_w4a16_linear(c.X, *c.dev, group_size=128, sym=False, activation="silu",
                                 gated=gated, residual=r, Y=r, out_dtype=r.dtype)
    assert got is r and torch.equal(r, want)


@pytest.mark.parametrize("m", [4, 150])
def test_no_rows_and_plain_product_agree(m):
    c = Case(m, 256, 96, 64, False, out="f32")
    assert gptq.gptq_w4a16_linear(c.X[:0], *c.dev, group_size=64, sym=False).shape == (0, 96)
    plain = gptq.gptq_w4a16_matmul(c.X.contiguous(), *c.dev, group_size=64, sym=False)
    c.check(plain)
    c.check(c.call())


@pytest.mark.parametrize("m", [3, 64, 65, 200])
def test_rows_are_their_own(m):
    """An infinity or a NaN in a row stays there, also where k is not whole chunks."""
    c = Case(m, 288, 150, 32, False, act="gelu", res="bf16")
    good = c.call()
    X = c.X.clone()
    X[m // 2, 287] = float("inf")
    X[m - 1, 0] = float("nan")
    got = gptq.gptq_w4a16_linear(X, *c.dev, group_size=32, sym=False, activation="gelu", residual=c.res)
    keep = [i for i in range(m) if i not in (m // 2, m - 1)]
    assert torch.equal(got[keep], good[keep])
    assert not bool(torch.isfinite(got[m - 1]).any())


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("m", [1, 70])
def test_activation_tails(act, m):
    """Zero weights: v is the bias, from the far tails to the far top."""
    v = np.concatenate([np.linspace(-90, 90, 721), [-1e4, 1e4, 0.0, -1e-30, 1e30, -1e30]]).astype(np.float32)
    n = len(v)
    X = torch.zeros((m, 32), dtype=torch.bfloat16, device=DEV)
    Q = torch.zeros((n, 4), dtype=torch.int32, device=DEV)
    S = torch.ones((n, 1), dtype=torch.float16, device=DEV)
    Y = gptq.gptq_w4a16_linear(X, Q, S, None, group_size=32, sym=True, activation=act,
                               bias=torch.from_numpy(v).to(DEV), out_dtype=torch.float32)
    import oracle
    with np.errstate(over="ignore"):
        want = oracle.activate(v, act)
    # the oracle's own tanh and erf cancel in the lower tail: held to their size there
    got = f64(Y)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want[None]) <= 40 * 2.0 ** -24 * np.abs(want) + 8 * 2.0 ** -24 + 1e-14 * np.abs(v))
    assert np.all(np.abs(got[:, v < -40]) <= 1e-12)


@pytest.mark.parametrize("off", [0, 1, 3])
def test_scales_at_any_address(off):
    """Rows of scales at addresses of 2 bytes, with an odd number of groups and an even one."""
    for d_in in (96, 256):
        c = Case(70, d_in, 140, 32, False, act="none", out="f32")
        Q, S, Z = c.dev
        room = torch.zeros(2 * S.numel() + 32, dtype=torch.int16, device=DEV)
        s = room[off:off + S.numel()].view(S.shape)
        z = room[S.numel() + 16 + off:2 * S.numel() + 16 + off].view(S.shape)
        s.copy_(S), z.copy_(Z)
        c.check(gptq.gptq_w4a16_linear(c.X, Q, s, z, group_size=32, sym=False, out_dtype=torch.float32))


@pytest.mark.parametrize("m", [1, 5, 40, 100])
@pytest.mark.parametrize("g,d_in", [(32, 672), (64, 1088), (128, 1664), (32, 1120)])
def test_weight_rows_are_their_own(m, g, d_in):
    """A row of weights whose scales are NaN spoils its own column alone, whatever the number of
    groups to a row divides by; the last rows' scales end where the array ends."""
    c = Case(m, d_in, 37, g, False)
    want = c.call()
    Q, S, Z = c.dev
    for row in (0, 17, 36):
        bad = S.clone()
        bad.view(torch.float16)[row] = float("nan")
        got = gptq.gptq_w4a16_linear(c.X, Q, bad, Z, group_size=g, sym=False)
        assert bool(torch.isnan(got[:, row]).all())
        keep = [n for n in range(37) if n != row]
        assert torch.equal(got[:, keep], want[:, keep])


@pytest.mark.parametrize("m", [1, 33, 65, 333])
def test_captured_and_replayed(m):
    c = Case(m, 4096, 264, 128, False, act="silu", gated=True, res="bf16", bias="bf16")
    Y = torch.empty((m, 132), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(max(1, gptq.gptq_w4a16_linear_workspace(m, 264, 4096, 128, True)), dtype=torch.uint8,
                     device=DEV)
    want = c.call().cpu()
    for (got,) in replayed(lambda: c.call(Y=Y, ws=ws), [Y]):
        assert torch.equal(got, want)


def test_two_calls_at_once():
    """On two streams, each with its own workspace."""
    cs = [Case(m, 4096, 520, 128, False, act="gelu", seed=m) for m in (40, 200)]
    want = [c.call() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        got = [c.call(stream=s) for c, s in zip(cs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_large_offsets():
    """X, Y and residual whose last rows lie past 2^31 elements."""
    m, ld = 300, 1 << 23
    c = Case(m, 64, 72, 64, False, act="silu", res="bf16")
    X = torch.zeros((m, ld), dtype=torch.bfloat16, device=DEV)[:, :64]
    Y = torch.zeros((m, ld), dtype=torch.bfloat16, device=DEV)[:, :72]
    X.copy_(c.X), Y.copy_(c.res)
    gptq.gptq_w4a16_linear(X, *c.dev, group_size=64, sym=False, activation="silu", residual=Y, Y=Y)
    c.check(Y)


@pytest.mark.parametrize("case", ["activation", "odd gate", "bias", "bias type", "residual", "Y", "Y type",
                                  "out_dtype", "qweight", "zeros", "X", "workspace", "host bias",
                                  "in place, two types"])
def test_refuses(case):
    c = Case(4, 256, 64, 128, False, bias="bf16")
    kw, X, dev = {}, c.X, list(c.dev)
    if case == "activation":
        kw["activation"] = "tanh"
    elif case == "odd gate":
        dev = [t[:63] for t in dev]
        kw.update(gated=True, bias=None)
    elif case == "bias":
        kw["bias"] = torch.zeros(63, device=DEV)
    elif case == "bias type":
        kw["bias"] = torch.zeros(64, dtype=torch.float16, device=DEV)
    elif case == "residual":
        kw["residual"] = torch.zeros((4, 63), device=DEV)
    elif case == "Y":
        kw["Y"] = torch.zeros((4, 65), dtype=torch.bfloat16, device=DEV)
    elif case == "Y type":
        kw["Y"] = torch.zeros((4, 64), device=DEV)
    elif case == "out_dtype":
        kw["out_dtype"] = torch.float16
    elif case == "qweight":
        dev[0] = dev[0][:, :-1]
    elif case == "zeros":
        dev[2] = None
    elif case == "X":
        X = X.float()
    elif case == "workspace":
        c = Case(100, 8192, 64, 128, False)
        X, dev = c.X, list(c.dev)
        assert gptq.gptq_w4a16_linear_workspace(100, 64, 8192, 128) > 16
        kw.update(ws=torch.zeros(16, dtype=torch.uint8, device=DEV), bias=None)
    elif case == "host bias":
        kw["bias"] = torch.zeros(64)
    elif case == "in place, two types":
        r = torch.zeros((4, 64), device=DEV)
        kw.update(residual=r, Y=r.view(torch.bfloat16)[:, :64])
    a = dict(group_size=128, sym=False, bias=c.bias) | kw
    with pytest.raises((ValueError, gptq.GPTQError)):
        gptq.gptq_w4a16_linear(X, *dev, **a)
