"""What the calls that complete a decoder block refuse.  CPU only: the library's own checks
return before anything is enqueued (the pointers are never followed), and the binding's
raise before the library is called."""
import os

import pytest
import torch

from post_weight_quantization_syrk_amd import gptq

A = 0x1000  # 256-byte aligned, never followed
OK, EINVAL, EUNSUP = gptq.GPTQ_OK, gptq.GPTQ_EINVAL, gptq.GPTQ_EUNSUPPORTED
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(gptq.LIB_PATH):
        pytest.skip("library not built")
    return gptq.lib()


def linear(L, **kw):
    a = dict(X=A, m=4, ldx=256, qw=A, s=A, z=A, d_out=8, d_in=256, g=128, sym=0, bias=A, bt=0, act=2,
             gated=0, res=A, rt=1, ldr=8, Y=A, yt=1, ldy=8, ws=A, ws_bytes=BIG) | kw
    return L.gptq_w4a16_linear(*a.values(), None)


LINEAR = [
    (dict(m=-1), EINVAL), (dict(m=(1 << 30) + 1), EINVAL),
    (dict(d_out=0), EINVAL), (dict(d_out=(1 << 30) + 1), EINVAL),
    (dict(d_in=0), EINVAL), (dict(d_in=65568, ldx=65568, g=32), EINVAL), (dict(d_in=-256), EINVAL),
    (dict(d_in=264, ldx=272, g=-1), EUNSUP),
    (dict(g=0), EINVAL), (dict(g=-2), EINVAL), (dict(g=96), EINVAL), (dict(g=256), EUNSUP), (dict(g=16), EUNSUP),
    (dict(sym=2), EINVAL), (dict(sym=-1), EINVAL),
    (dict(gated=2), EINVAL), (dict(gated=-1), EINVAL), (dict(gated=1, d_out=7), EINVAL),
    (dict(act=-1), EINVAL), (dict(act=5), EINVAL),
    (dict(bt=2), EINVAL), (dict(rt=2), EINVAL), (dict(yt=2), EINVAL), (dict(yt=-1), EINVAL),
    (dict(ldx=240), EINVAL), (dict(ldx=260), EINVAL), (dict(X=None), EINVAL), (dict(X=A + 8), EINVAL),
    (dict(ldx=(1 << 23) + 8), EUNSUP),
    (dict(qw=None), EINVAL), (dict(qw=A + 4), EINVAL), (dict(s=None), EINVAL), (dict(s=A + 1), EINVAL),
    (dict(z=None), EINVAL), (dict(z=A + 1), EINVAL),
    (dict(Y=None, res=None), EINVAL), (dict(Y=A + 2, res=None), EINVAL), (dict(Y=A + 1, yt=0, res=None), EINVAL),
    (dict(ldy=7), EINVAL), (dict(ldr=7), EINVAL), (dict(gated=1, ldy=3, res=None), EINVAL),
    (dict(bias=A + 1), EINVAL), (dict(bias=A + 2, bt=1), EINVAL), (dict(res=A + 2), EINVAL),
    (dict(ldr=9), EINVAL), (dict(rt=0), EINVAL),      # in place with two strides, or two types
    (dict(m=0, X=None, Y=None), OK), (dict(m=0, g=96), EINVAL), (dict(m=0, bias=None, bt=9), OK),
]


@pytest.mark.parametrize("kw,want", LINEAR)
def test_linear_refuses(L, kw, want):
    assert linear(L, **kw) == want


def test_linear_workspace_is_required_where_it_is_reported(L):
    asked = 0
    for m in (1, 2, 16, 33, 64, 65, 100, 515, 4096):
        for d_out, d_in in ((64, 4096), (4096, 4096), (4098, 11008), (22016, 4096)):
            for gated in (0, 1):
                need = gptq.gptq_w4a16_linear_workspace(m, d_out, d_in, 128, bool(gated))
                asked += need > 0
                kw = dict(m=m, d_out=d_out, d_in=d_in, ldx=d_in, gated=gated, ldy=d_out, ldr=d_out)
                if need:
                    assert linear(L, **kw, ws_bytes=need - 1) == EINVAL
                    assert linear(L, **kw, ws=None, ws_bytes=need) == EINVAL
                    assert linear(L, **kw, ws=A + 64, ws_bytes=need) == EINVAL
    assert asked
    assert gptq.gptq_w4a16_linear_workspace(0, 64, 4096, 128) == 0
    assert gptq.gptq_w4a16_linear_workspace(100, 64, 4000, 128) == 0
    assert gptq.gptq_w4a16_linear_workspace(100, 63, 4096, 128, True) == 0


def rope(L, **kw):
    a = dict(Q=A, ldq=512, hsq=64, K=A, ldk=256, hsk=64, V=A, ldv=256, hsv=64, x=0, m=4, hq=8, hk=4, hd=64,
             pos=A, freq=A, rot=64, inter=0, qw=A, kw=A, wt=0, eps=1e-6, slots=None, rows=4,
             Qo=A, ldqo=512, hsqo=64, Ko=A, ldko=256, hsko=64, Vo=A, ldvo=256, hsvo=64) | kw
    return L.gptq_qk_norm_rope(*a.values(), None)


ROPE = [
    (dict(m=-1), EINVAL), (dict(m=(1 << 30) + 1), EINVAL), (dict(hq=0), EINVAL), (dict(hk=0), EINVAL),
    (dict(hd=0), EINVAL), (dict(hd=-8), EINVAL), (dict(rot=-16), EINVAL), (dict(rot=80), EINVAL),
    (dict(rot=31), EINVAL), (dict(rows=-1), EINVAL),
    (dict(x=2), EINVAL), (dict(inter=2), EINVAL), (dict(wt=2), EINVAL),
    (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL),
    (dict(hd=60, rot=32), EUNSUP), (dict(hd=264), EUNSUP), (dict(rot=24), EUNSUP), (dict(hq=65537), EUNSUP),
    (dict(V=None), EINVAL), (dict(Vo=None), EINVAL),
    (dict(Q=None), EINVAL), (dict(K=None), EINVAL), (dict(Qo=None), EINVAL), (dict(Ko=None), EINVAL),
    (dict(pos=None), EINVAL), (dict(freq=None), EINVAL), (dict(pos=A + 2), EINVAL), (dict(freq=A + 4), EINVAL),
    (dict(rows=3), EINVAL), (dict(slots=A + 4), EINVAL),
    (dict(Q=A + 8), EINVAL), (dict(K=A + 8), EINVAL), (dict(V=A + 8), EINVAL), (dict(Qo=A + 8), EINVAL),
    (dict(Ko=A + 8), EINVAL), (dict(Vo=A + 8), EINVAL), (dict(qw=A + 1), EINVAL), (dict(kw=A + 2, wt=1), EINVAL),
    (dict(ldq=-8), EINVAL), (dict(ldq=516), EINVAL), (dict(hsk=68), EINVAL), (dict(ldv=1 << 23), EUNSUP),
    (dict(hsq=1 << 40), EUNSUP),
    # outputs whose values share places
    (dict(ldqo=504), EINVAL), (dict(hsqo=56), EINVAL), (dict(ldko=0), EINVAL), (dict(hsvo=0), EINVAL),
    (dict(ldqo=64, hsqo=248), EINVAL), (dict(slots=A, rows=9, ldko=64, hsko=256), EINVAL),
    (dict(m=0), OK), (dict(m=0, Q=None, Ko=None), OK),
    (dict(m=0, V=None), OK),                          # no tokens, with a cache to write to
    (dict(slots=A, rows=(1 << 38) + 1), EINVAL), (dict(m=1 << 29, rows=1 << 29), EUNSUP),
]


@pytest.mark.parametrize("kw,want", ROPE)
def test_rope_refuses(L, kw, want):
    assert rope(L, **kw) == want


def attention(L, **kw):
    a = dict(Q=A, ldq=512, hsq=64, K=A, ldk=256, hsk=64, V=A, ldv=256, hsv=64, tq=100, rows=200, batch=3, hq=8,
             hk=4, hd=64, cu=A, start=A, len=A, longest=200, causal=1, scale=0.125, out=A, ldo=512, hso=64,
             ws=A, ws_bytes=BIG) | kw
    return L.gptq_attention(*a.values(), None)


ATTENTION = [
    (dict(tq=-1), EINVAL), (dict(tq=(1 << 30) + 1), EINVAL), (dict(batch=-1), EINVAL),
    (dict(batch=(1 << 30) + 1), EINVAL), (dict(rows=-1), EINVAL), (dict(longest=-1), EINVAL),
    (dict(hq=0), EINVAL), (dict(hk=0), EINVAL), (dict(hd=0), EINVAL), (dict(hq=6), EINVAL),
    (dict(hq=65540), EUNSUP), (dict(hd=60), EUNSUP), (dict(hd=264), EUNSUP),
    (dict(batch=1 << 24), EUNSUP), (dict(tq=1 << 29), EUNSUP),
    (dict(causal=2), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL),
    (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(scale=1e-46), EINVAL),
    (dict(rows=(1 << 38) + 1), EINVAL), (dict(batch=1 << 21), EUNSUP), (dict(tq=1 << 26, hq=64), EUNSUP),
    (dict(start=None), EINVAL), (dict(len=None), EINVAL),
    (dict(Q=None), EINVAL), (dict(K=None), EINVAL), (dict(V=None), EINVAL), (dict(out=None), EINVAL),
    (dict(cu=None), EINVAL), (dict(Q=A + 8), EINVAL), (dict(K=A + 2), EINVAL), (dict(V=A + 4), EINVAL),
    (dict(out=A + 8), EINVAL), (dict(cu=A + 2), EINVAL), (dict(start=A + 4), EINVAL), (dict(len=A + 2), EINVAL),
    (dict(ldq=-512), EINVAL), (dict(ldk=260), EINVAL), (dict(hsv=4), EINVAL), (dict(ldk=1 << 23), EUNSUP),
    (dict(ldo=504), EINVAL), (dict(hso=56), EINVAL), (dict(ldo=0), EINVAL),
    (dict(ldo=64, hso=64 * 99), EINVAL),
    (dict(tq=0), OK), (dict(batch=0), OK), (dict(tq=0, Q=None, out=None, cu=None), OK),
]


@pytest.mark.parametrize("kw,want", ATTENTION)
def test_attention_refuses(L, kw, want):
    assert attention(L, **kw) == want


def test_attention_workspace_is_required_where_it_is_reported(L):
    asked = 0
    for tq, batch in ((1, 1), (4, 1), (64, 64), (300, 1), (16384, 1)):
        for hq, hk, hd in ((8, 1, 128), (32, 8, 128), (4, 4, 256)):
            need = gptq.gptq_attention_workspace(tq, batch, hq, hk, hd, 20000)
            asked += need > 0
            if need:
                kw = dict(tq=tq, batch=batch, hq=hq, hk=hk, hd=hd, rows=20000, longest=20000, ldq=hq * hd, hsq=hd,
                          ldo=hq * hd, hso=hd)
                assert attention(L, **kw, ws_bytes=need - 1) == EINVAL
                assert attention(L, **kw, ws=None, ws_bytes=need) == EINVAL
                assert attention(L, **kw, ws=A + 64, ws_bytes=need) == EINVAL
    assert asked
    assert gptq.gptq_attention_workspace(0, 1, 8, 8, 64, 100) == 0
    assert gptq.gptq_attention_workspace(4, 1, 8, 8, 60, 100) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    q = torch.zeros((8, 32), dtype=torch.int32)
    s = torch.zeros((8, 2), dtype=torch.int16)
    h = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        gptq.gptq_w4a16_linear(x, q, s, s, group_size=128, sym=False)
    with pytest.raises(ValueError, match="GPU"):
        gptq.gptq_qk_norm_rope(h, h, positions=None, inv_freq=None)
    with pytest.raises(ValueError, match="GPU"):
        gptq.gptq_attention(h, h, h, cu_q=torch.tensor([0, 2], dtype=torch.int32))
