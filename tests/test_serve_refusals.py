"""What the calls that run a quantized layer refuse.  CPU only: the library's own checks
return before anything is enqueued (the pointers are never followed), and the binding's
raise before the library is called."""
import ctypes
import os

import pytest
import torch

from post_weight_quantization_syrk_amd import gptq

P = ctypes.c_void_p
A = 0x1000  # 256-byte aligned, never followed
OK, EINVAL, EUNSUP = gptq.GPTQ_OK, gptq.GPTQ_EINVAL, gptq.GPTQ_EUNSUPPORTED


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(gptq.LIB_PATH):
        pytest.skip("library not built")
    return gptq.lib()


def matvec(L, **kw):
    a = dict(X=A, m=4, ldx=256, qw=A, s=A, z=A, d_out=8, d_in=256, g=128, sym=0, Y=A,
             ws=A, ws_bytes=1 << 40) | kw
    return L.gptq_w4a16_matvec(*a.values(), None)


def w4a8(L, **kw):
    a = dict(X=A, xs=A, m=4, ldx=256, qw=A, s=A, z=A, d_out=8, d_in=256, g=128, sym=0, Y=A,
             ws=A, ws_bytes=1 << 40) | kw
    return L.gptq_w4a8_matmul(*a.values(), None)


def norm(L, **kw):
    a = dict(X=A, x=1, ldx=256, R=A, r=0, ldr=256, Ro=A, ldro=256, w=A, wt=0, eps=1e-6, m=4, d=256,
             out=A, o=2, ldo=256, s=A) | kw
    return L.gptq_add_rmsnorm(*a.values(), None)


W4 = [
    (dict(m=-1), EINVAL), (dict(m=(1 << 30) + 1), EINVAL),
    (dict(d_out=0), EINVAL), (dict(d_out=(1 << 30) + 1), EINVAL),
    (dict(d_in=0), EINVAL), (dict(d_in=65568, ldx=65568, g=32), EINVAL),
    (dict(d_in=-256), EINVAL),
    (dict(d_in=264, ldx=272, g=-1), EUNSUP),     # d_in % 32
    (dict(g=0), EINVAL), (dict(g=-2), EINVAL), (dict(g=96), EINVAL),
    (dict(g=256), EUNSUP), (dict(g=16), EUNSUP),
    (dict(sym=2), EINVAL), (dict(sym=-1), EINVAL),
    (dict(ldx=240), EINVAL), (dict(ldx=260), EINVAL), (dict(ldx=0), EINVAL),
    (dict(X=None), EINVAL), (dict(X=A + 8), EINVAL),
    (dict(qw=None), EINVAL), (dict(qw=A + 4), EINVAL),
    (dict(s=None), EINVAL), (dict(s=A + 1), EINVAL),
    (dict(z=None), EINVAL), (dict(z=A + 1), EINVAL),
    (dict(Y=None), EINVAL), (dict(Y=A + 2), EINVAL),
    (dict(m=0, X=None, Y=None), OK),
    (dict(m=0, g=96), EINVAL),
]


@pytest.mark.parametrize("kw,want", W4)
def test_both_products_refuse(L, kw, want):
    assert matvec(L, **kw) == want
    assert w4a8(L, **kw) == want


def test_products_own_refusals(L):
    assert matvec(L, m=gptq.GPTQ_MATVEC_MAX_M + 1) == EUNSUP
    assert w4a8(L, xs=None) == EINVAL
    assert w4a8(L, xs=A + 2) == EINVAL
    assert w4a8(L, ldx=264) == EINVAL  # a multiple of 8, not of 16
    assert gptq.gptq_w4a8_workspace(0, 64, 256, 128) == 0
    assert gptq.gptq_w4a8_workspace(4, 64, 250, 128) == 0
    assert gptq.gptq_w4a8_workspace(4, 0, 256, 128) == 0


@pytest.mark.parametrize("call,query,ms", [
    (matvec, gptq.gptq_w4a16_matvec_workspace, (1, 2, 5, 16, 17, 40, 64)),
    (w4a8, gptq.gptq_w4a8_workspace, (1, 2, 16, 40, 64, 65, 100, 300, 515, 1000, 4096)),
])
def test_workspace_is_required_where_it_is_reported(L, call, query, ms):
    asked = shapes = 0
    for m in ms:
        for d_out, d_in in ((64, 4096), (512, 12288), (4096, 4096), (4099, 11008), (11008, 4096)):
            need = query(m, d_out, d_in, 128 if d_in % 128 == 0 else 32)
            shapes += 1
            asked += need > 0
            if need:
                kw = dict(m=m, d_out=d_out, d_in=d_in, ldx=d_in)
                assert call(L, **kw, ws_bytes=need - 1) == EINVAL
                assert call(L, **kw, ws=None, ws_bytes=need) == EINVAL
                assert call(L, **kw, ws=A + 64, ws_bytes=need) == EINVAL
    print(f"{asked} of {shapes} shapes ask for a workspace")
    assert asked
    assert query(0, 64, 4096, 128) == 0 and query(4, 64, 4000, 128) == 0


NORM = [
    (dict(m=-1), EINVAL), (dict(m=(1 << 30) + 1), EINVAL),
    (dict(d=0), EINVAL), (dict(d=65537, ldx=70000, ldr=70000, ldro=70000, ldo=70000), EINVAL),
    (dict(x=2), EINVAL), (dict(x=7), EINVAL), (dict(r=2), EINVAL), (dict(r=-1), EINVAL),
    (dict(wt=2), EINVAL), (dict(o=1), EUNSUP), (dict(o=3), EINVAL), (dict(o=-1), EINVAL),
    (dict(eps=-1e-6), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL),
    (dict(R=None), EINVAL),                       # R_out without R
    (dict(ldx=255), EINVAL), (dict(ldr=255), EINVAL), (dict(ldro=255), EINVAL),
    (dict(ldo=255), EINVAL),
    (dict(ldr=264), EINVAL),                      # in place with two leading dimensions
    (dict(X=None), EINVAL), (dict(w=None), EINVAL), (dict(out=None), EINVAL),
    (dict(s=None), EINVAL),
    (dict(X=A + 2), EINVAL), (dict(X=A + 1, x=0), EINVAL), (dict(R=A + 1, Ro=None), EINVAL),
    (dict(Ro=A + 1), EINVAL), (dict(R=A + 2, Ro=None, r=1), EINVAL),
    (dict(w=A + 1), EINVAL), (dict(w=A + 2, wt=1), EINVAL), (dict(out=A + 1, o=0), EINVAL),
    (dict(s=A + 2), EINVAL),
    (dict(m=0), OK), (dict(m=0, X=None, out=None, s=None), OK),
    (dict(m=0, r=5, R=None, Ro=None), OK),        # r_dtype is ignored without R
]


@pytest.mark.parametrize("kw,want", NORM)
def test_add_rmsnorm_refuses(L, kw, want):
    assert norm(L, **kw) == want


def test_existing_calls_refuse_the_8_bit_type(L):
    assert L.gptq_hessian_accumulate(A, 16, A, gptq.GPTQ_I8, 10, 16, A, 1 << 30, None) == EINVAL


def test_binding_refuses_host_tensors_and_types():
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    q = torch.zeros((8, 32), dtype=torch.int32)
    s = torch.zeros((8, 2), dtype=torch.int16)
    with pytest.raises(ValueError, match="GPU"):
        gptq.gptq_w4a16_matvec(x, q, s, s, group_size=128, sym=False)
    with pytest.raises(ValueError, match="GPU"):
        gptq.gptq_w4a16_matvec(x.float(), q, s, s, group_size=128, sym=False)
    with pytest.raises(ValueError, match="GPU"):
        gptq.gptq_w4a8_matmul(x.to(torch.int8), torch.zeros(2), q, s, s, group_size=128, sym=False)
    with pytest.raises(ValueError, match="GPU"):
        gptq.gptq_add_rmsnorm(x, torch.zeros(256, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="GPU"):
        gptq.gptq_add_rmsnorm(x.half(), torch.zeros(256, dtype=torch.bfloat16))
