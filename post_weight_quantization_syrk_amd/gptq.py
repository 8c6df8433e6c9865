"""Thin ctypes binding of libgptq_mi355x.so (C ABI in include/gptq.h).

Argument marshalling only: every step of the path runs in the HIP library.
PyTorch provides device memory (tensors, workspaces) and the stream.  The
functions keep the C names; tensors replace raw pointers, and outputs that the
caller does not pass in are allocated here with torch.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgptq_mi355x.so")

GPTQ_OK, GPTQ_EINVAL, GPTQ_EUNSUPPORTED, GPTQ_EHIP, GPTQ_ENOTSPD = range(5)
GPTQ_BF16, GPTQ_F32, GPTQ_I8 = 0, 1, 2
GPTQ_MATVEC_MAX_M = 64

_lib = None


class GPTQError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {strerror(status)} (status {status})")
        self.status = status


class SyncTimeoutError(GPTQError):
    def __init__(self, where: str):
        RuntimeError.__init__(self, f"{where}: a bounded wait between workgroups expired "
                                    "(dev_status -1); the factorization did not complete")
        self.status = GPTQ_EHIP


def _raise_status(st: int, where: str):
    if st > 0:
        raise NotSPDError(st)
    if st < 0:
        raise SyncTimeoutError(where)


class NotSPDError(GPTQError):
    def __init__(self, pivot: int):
        RuntimeError.__init__(self, f"gptq_prepare_hinv: Hessian not positive definite "
                                    f"(pivot index {pivot - 1})")
        self.status = GPTQ_ENOTSPD
        self.pivot = pivot


def lib() -> ctypes.CDLL:
    """Load the HIP library; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                           "or python -m post_weight_quantization_syrk_amd.build")
    L = ctypes.CDLL(LIB_PATH)
    P, I64, I, SZ, D = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_double
    sig = {
        "gptq_hessian_accumulate": (I, [P, I64, P, I, I64, I64, P, SZ, P]),
        "gptq_hessian_workspace": (SZ, [I64, I64, I]),
        "gptq_hessian_accumulate_noalloc": (I, [P, I64, P, I, I64, I64, P]),
        "gptq_noalloc_scratch_bytes": (SZ, []),
        "gptq_prepare_hinv": (I, [P, I64, D, P, P, P, P, SZ, P]),
        "gptq_prepare_workspace": (SZ, [I64]),
        "gptq_quantize_layer": (I, [P, I, I64, I64, P, P, I, I, I, I, P, P, P, P, P, SZ, P]),
        "gptq_quantize_workspace": (SZ, [I64, I64, I]),
        "gptq_pack": (I, [P, P, P, I64, I64, I, I, I, P, P, P, P]),
        "gptq2d_round": (I, [P, P, P, I64, P, P, SZ, P]),
        "gptq_w4a16_matmul": (I, [P, I64, I64, P, P, P, I64, I64, I, I, P, P]),
        "gptq_w4a16_matvec": (I, [P, I64, I64, P, P, P, I64, I64, I, I, P, P, SZ, P]),
        "gptq_w4a16_matvec_workspace": (SZ, [I64, I64, I64, I]),
        "gptq_w4a8_matmul": (I, [P, P, I64, I64, P, P, P, I64, I64, I, I, P, P, SZ, P]),
        "gptq_w4a8_workspace": (SZ, [I64, I64, I64, I]),
        "gptq_add_rmsnorm": (I, [P, I, I64, P, I, I64, P, I64, P, I, D, I64, I64, P, I, I64, P,
                                 P]),
        "gptq_quantize_layers": (I, [P, P, I, I, I64, P, P, I, I, I, I, P, P, P, P, P, SZ, P]),
        "gptq_act_order": (I, [P, I, I64, I64, I64, P, P, P, SZ, P]),
        "gptq_act_order_workspace": (SZ, [I64, I64]),
        "gptq_prepare_hinv_perm": (I, [P, I64, D, P, P, P, P, P, SZ, P]),
        "gptq_quantize_layer_perm": (I, [P, I, I64, I64, P, P, P, I, I, I, I, I, P, P, P, P, P,
                                         P, SZ, P]),
        "gptq_quantize_perm_workspace": (SZ, [I64, I64, I]),
        "gptq2d_workspace": (SZ, [I64]),
        "gptq_strerror": (ctypes.c_char_p, [I]),
        "gptq_abi_version": (I, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def strerror(status: int) -> str:
    return lib().gptq_strerror(status).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(status: int, where: str):
    if status != GPTQ_OK:
        raise GPTQError(status, where)


def _empty(stream, *args, **kw) -> torch.Tensor:
    """torch.empty, allocated on the stream the call will launch on: the
    caching allocator then hands the block out again only in that stream's
    order, so a buffer dropped when the call returns (its scratch) cannot be
    reused while the call's kernels still run on a stream other than the
    current one."""
    if stream is None:
        return torch.empty(*args, **kw)
    with torch.cuda.stream(stream):
        return torch.empty(*args, **kw)


def _workspace(nbytes: int, device, stream=None) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    return _empty(stream, nbytes, dtype=torch.uint8, device=device)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GPTQ_BF16
    if t.dtype == torch.float32:
        return GPTQ_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


# --------------------------------------------------------------------------
def gptq_hessian_workspace(d: int, n_tokens: int, x_dtype: int) -> int:
    return int(lib().gptq_hessian_workspace(d, n_tokens, x_dtype))


def gptq_hessian_accumulate(H: torch.Tensor, X: torch.Tensor, ws: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """H (lower triangle) += 2 X^T X.  H [d, d] fp32; X [n, d] (row stride may exceed d)."""
    d = H.shape[0]
    if X.dim() != 2 or X.stride(1) != 1 or H.dtype != torch.float32 or not H.is_contiguous():
        raise ValueError("H must be contiguous fp32 [d, d]; X a row-major [n, >=d] matrix")
    if X.shape[1] < d:
        raise ValueError("X has fewer columns than d")
    xd = _dtype_code(X)
    n = X.shape[0]
    need = gptq_hessian_workspace(d, n, xd)
    if ws is None:
        ws = _workspace(need, H.device, stream)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().gptq_hessian_accumulate(_ptr(H), d, _ptr(X), xd, n, X.stride(0), _ptr(ws),
                                         nbytes, _stream(stream)), "gptq_hessian_accumulate")
    return H


def gptq_hessian_accumulate_noalloc(H: torch.Tensor, X: torch.Tensor, stream=None) -> torch.Tensor:
    """H (lower triangle) += 2 X^T X with the library's fixed per-GPU scratch: no
    device memory is allocated by this call (nor by the library)."""
    d = H.shape[0]
    if X.dim() != 2 or X.stride(1) != 1 or H.dtype != torch.float32 or not H.is_contiguous():
        raise ValueError("H must be contiguous fp32 [d, d]; X a row-major [n, >=d] matrix")
    if X.shape[1] < d:
        raise ValueError("X has fewer columns than d")
    _check(lib().gptq_hessian_accumulate_noalloc(_ptr(H), d, _ptr(X), _dtype_code(X), X.shape[0],
                                                 X.stride(0), _stream(stream)),
           "gptq_hessian_accumulate_noalloc")
    return H


def gptq_noalloc_scratch_bytes() -> int:
    return int(lib().gptq_noalloc_scratch_bytes())


def gptq_prepare_workspace(d: int) -> int:
    return int(lib().gptq_prepare_workspace(d))


def gptq_prepare_hinv(H: torch.Tensor, damp: float = 0.01, U: torch.Tensor | None = None,
                      dead: torch.Tensor | None = None, status: torch.Tensor | None = None,
                      ws: torch.Tensor | None = None, stream=None, check: bool = True):
    """Damp H in place and compute U (U^T U = H^-1).  Returns (U, dead, status).

    With check=True the stream is synchronised and a breakdown raises NotSPDError.
    """
    d = H.shape[0]
    dev = H.device
    if U is None:
        U = _empty(stream, (d, d), dtype=torch.float32, device=dev)
    if dead is None:
        dead = _empty(stream, d, dtype=torch.uint8, device=dev)
    if status is None:
        status = _empty(stream, 1, dtype=torch.int32, device=dev)
    if ws is None:
        ws = _workspace(gptq_prepare_workspace(d), dev, stream)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().gptq_prepare_hinv(_ptr(H), d, float(damp), _ptr(U), _ptr(dead), _ptr(status),
                                   _ptr(ws), nbytes, _stream(stream)), "gptq_prepare_hinv")
    if check:
        (torch.cuda.current_stream() if stream is None else stream).synchronize()
        _raise_status(int(status.item()), "gptq_prepare_hinv")
    return U, dead, status


def gptq_quantize_workspace(d_out: int, d_in: int, block: int = 128) -> int:
    return int(lib().gptq_quantize_workspace(d_out, d_in, block))


def n_groups_for(d_in: int, group_size: int) -> int:
    return 1 if group_size == -1 else d_in // group_size


def gptq_quantize_layer(W: torch.Tensor, U: torch.Tensor, dead: torch.Tensor | None = None, *,
                        bits: int = 4, group_size: int = 128, sym: bool = False,
                        block: int = 128, codes=None, scales=None, zeros=None, loss_rows=None,
                        want_loss: bool = True, ws=None, stream=None):
    """Returns (codes uint8, scales fp32, zeros fp32, loss_rows fp32 or None)."""
    d_out, d_in = W.shape
    dev = W.device
    if not W.is_contiguous() or not U.is_contiguous():
        raise ValueError("W and U must be contiguous")
    ng = n_groups_for(d_in, group_size) if group_size > 0 or group_size == -1 else 1
    if codes is None:
        codes = _empty(stream, (d_out, d_in), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = _empty(stream, (d_out, max(ng, 1)), dtype=torch.float32, device=dev)
    if zeros is None:
        zeros = _empty(stream, (d_out, max(ng, 1)), dtype=torch.float32, device=dev)
    if loss_rows is None and want_loss:
        loss_rows = _empty(stream, d_out, dtype=torch.float32, device=dev)
    if ws is None:
        ws = _workspace(gptq_quantize_workspace(d_out, d_in, block), dev, stream)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().gptq_quantize_layer(_ptr(W), _dtype_code(W), d_out, d_in, _ptr(U), _ptr(dead),
                                     bits, group_size, int(bool(sym)), block, _ptr(codes),
                                     _ptr(scales), _ptr(zeros), _ptr(loss_rows), _ptr(ws),
                                     nbytes, _stream(stream)), "gptq_quantize_layer")
    return codes, scales, zeros, loss_rows


# -------------------------------------------------- layers sharing one Hessian
def gptq_quantize_layers(Ws: list, U: torch.Tensor, dead: torch.Tensor | None = None, *,
                         bits: int = 4, group_size: int = 128, sym: bool = False,
                         block: int = 128, want_loss: bool = True, ws=None, stream=None):
    """Quantize several matrices [d_out_i, d_in] that share U in one call.  Returns
    (codes, scales, zeros, loss_rows) stacked by rows in list order, and the list of
    per-matrix row slices."""
    if not Ws:
        raise ValueError("no matrices")
    d_in = Ws[0].shape[1]
    dt = _dtype_code(Ws[0])
    for w in Ws:
        if w.dim() != 2 or w.shape[1] != d_in or not w.is_contiguous() or _dtype_code(w) != dt:
            raise ValueError("matrices must be contiguous [d_out_i, d_in] of one dtype")
    dev = Ws[0].device
    rows = [int(w.shape[0]) for w in Ws]
    total = sum(rows)
    ng = n_groups_for(d_in, group_size) if group_size > 0 or group_size == -1 else 1
    codes = _empty(stream, (total, d_in), dtype=torch.uint8, device=dev)
    scales = _empty(stream, (total, max(ng, 1)), dtype=torch.float32, device=dev)
    zeros = _empty(stream, (total, max(ng, 1)), dtype=torch.float32, device=dev)
    loss_rows = _empty(stream, total, dtype=torch.float32, device=dev) if want_loss else None
    if ws is None:
        ws = _workspace(gptq_quantize_workspace(total, d_in, block), dev, stream)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    ptrs = (ctypes.c_void_p * len(Ws))(*[w.data_ptr() for w in Ws])
    dl = (ctypes.c_int64 * len(Ws))(*rows)
    _check(lib().gptq_quantize_layers(ptrs, dl, len(Ws), dt, d_in, _ptr(U), _ptr(dead), bits,
                                      group_size, int(bool(sym)), block, _ptr(codes),
                                      _ptr(scales), _ptr(zeros), _ptr(loss_rows), _ptr(ws),
                                      nbytes, _stream(stream)), "gptq_quantize_layers")
    offs, slices = 0, []
    for r in rows:
        slices.append(slice(offs, offs + r))
        offs += r
    return codes, scales, zeros, loss_rows, slices


# -------------------------------------------------- activation ordering
def gptq_act_order_workspace(d: int, n_tokens: int) -> int:
    return int(lib().gptq_act_order_workspace(d, n_tokens))


def gptq_act_order(X: torch.Tensor, d: int | None = None, perm=None, act_sum=None, ws=None,
                   stream=None):
    """perm [d] int32: columns by ascending sum_t |X[t, c]|, ties by index.
    Returns (perm, act_sum float64 or None)."""
    if X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be a row-major [n, >=d] matrix")
    d = X.shape[1] if d is None else d
    n = X.shape[0]
    if perm is None:
        perm = _empty(stream, d, dtype=torch.int32, device=X.device)
    if ws is None:
        ws = _workspace(gptq_act_order_workspace(d, n), X.device, stream)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().gptq_act_order(_ptr(X), _dtype_code(X), n, X.stride(0), d, _ptr(perm),
                                _ptr(act_sum), _ptr(ws), nbytes, _stream(stream)),
           "gptq_act_order")
    return perm, act_sum


def gptq_prepare_hinv_perm(H: torch.Tensor, perm: torch.Tensor | None, damp: float = 0.01,
                           U=None, dead=None, status=None, ws=None, stream=None,
                           check: bool = True):
    """gptq_prepare_hinv for H[perm][:, perm].  Returns (U, dead, status)."""
    d = H.shape[0]
    dev = H.device
    if perm is not None and (perm.dtype != torch.int32 or perm.numel() != d):
        raise ValueError("perm must be an int32 tensor of d entries")
    if U is None:
        U = _empty(stream, (d, d), dtype=torch.float32, device=dev)
    if dead is None:
        dead = _empty(stream, d, dtype=torch.uint8, device=dev)
    if status is None:
        status = _empty(stream, 1, dtype=torch.int32, device=dev)
    if ws is None:
        ws = _workspace(gptq_prepare_workspace(d), dev, stream)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().gptq_prepare_hinv_perm(_ptr(H), d, float(damp), _ptr(perm), _ptr(U), _ptr(dead),
                                        _ptr(status), _ptr(ws), nbytes, _stream(stream)),
           "gptq_prepare_hinv_perm")
    if check:
        (torch.cuda.current_stream() if stream is None else stream).synchronize()
        _raise_status(int(status.item()), "gptq_prepare_hinv_perm")
    return U, dead, status


def gptq_quantize_perm_workspace(d_out: int, d_in: int, block: int = 128) -> int:
    return int(lib().gptq_quantize_perm_workspace(d_out, d_in, block))


def gptq_quantize_layer_perm(W: torch.Tensor, U: torch.Tensor, dead: torch.Tensor | None,
                             perm: torch.Tensor | None, *, static_groups: bool = False,
                             bits: int = 4, group_size: int = 128, sym: bool = False,
                             block: int = 128, codes=None, scales=None, zeros=None, g_idx=None,
                             loss_rows=None, want_loss: bool = True, ws=None, stream=None):
    """Returns (codes uint8 in natural column order, scales, zeros, g_idx int32, loss_rows)."""
    d_out, d_in = W.shape
    dev = W.device
    if not W.is_contiguous() or not U.is_contiguous():
        raise ValueError("W and U must be contiguous")
    if perm is not None and (perm.dtype != torch.int32 or perm.numel() != d_in):
        raise ValueError("perm must be an int32 tensor of d_in entries")
    ng = n_groups_for(d_in, group_size) if group_size > 0 or group_size == -1 else 1
    if codes is None:
        codes = _empty(stream, (d_out, d_in), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = _empty(stream, (d_out, max(ng, 1)), dtype=torch.float32, device=dev)
    if zeros is None:
        zeros = _empty(stream, (d_out, max(ng, 1)), dtype=torch.float32, device=dev)
    if g_idx is None:
        g_idx = _empty(stream, d_in, dtype=torch.int32, device=dev)
    if loss_rows is None and want_loss:
        loss_rows = _empty(stream, d_out, dtype=torch.float32, device=dev)
    if ws is None:
        ws = _workspace(gptq_quantize_perm_workspace(d_out, d_in, block), dev, stream)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().gptq_quantize_layer_perm(_ptr(W), _dtype_code(W), d_out, d_in, _ptr(U),
                                          _ptr(dead), _ptr(perm), int(bool(static_groups)), bits,
                                          group_size, int(bool(sym)), block, _ptr(codes),
                                          _ptr(scales), _ptr(zeros), _ptr(g_idx),
                                          _ptr(loss_rows), _ptr(ws), nbytes, _stream(stream)),
           "gptq_quantize_layer_perm")
    return codes, scales, zeros, g_idx, loss_rows


def gptq_pack(codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None, *,
              bits: int, group_size: int, sym: bool, qweight=None, scales_f16=None,
              zeros_f16=None, stream=None):
    """Returns (qweight uint32 as int32 tensor, scales_f16 bits, zeros_f16 bits or None)."""
    d_out, d_in = codes.shape
    dev = codes.device
    words = (d_in * bits + 31) // 32
    ng = n_groups_for(d_in, group_size)
    if qweight is None:
        qweight = _empty(stream, (d_out, words), dtype=torch.int32, device=dev)
    if scales_f16 is None:
        scales_f16 = _empty(stream, (d_out, ng), dtype=torch.int16, device=dev)
    if zeros_f16 is None and not sym:
        zeros_f16 = _empty(stream, (d_out, ng), dtype=torch.int16, device=dev)
    _check(lib().gptq_pack(_ptr(codes), _ptr(scales), _ptr(zeros), d_out, d_in, bits, group_size,
                           int(bool(sym)), _ptr(qweight), _ptr(scales_f16), _ptr(zeros_f16),
                           _stream(stream)), "gptq_pack")
    return qweight, scales_f16, zeros_f16


# --------------------------------------------------------------------------
def gptq2d_workspace(n: int) -> int:
    return int(lib().gptq2d_workspace(n))


def gptq2d_round(Y: torch.Tensor, left_basis: torch.Tensor, right_basis: torch.Tensor,
                 Z: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """Two-sided rounding of Y [n, n] float64 under upper-triangular bases; returns Z (float64
    integers).  Only the bases' upper triangles are read."""
    n = Y.shape[0]
    for name, t in (("Y", Y), ("left_basis", left_basis), ("right_basis", right_basis)):
        if t.shape != (n, n) or t.dtype != torch.float64 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float64 [n, n] tensor")
    if Z is None:
        Z = _empty(stream, (n, n), dtype=torch.float64, device=Y.device)
    if ws is None:
        ws = _workspace(gptq2d_workspace(n), Y.device, stream)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().gptq2d_round(_ptr(Y), _ptr(left_basis), _ptr(right_basis), n, _ptr(Z), _ptr(ws),
                              nbytes, _stream(stream)), "gptq2d_round")
    return Z


# --------------------------------------------------------------------------
def gptq_w4a16_matmul(X: torch.Tensor, qweight: torch.Tensor, scales_f16: torch.Tensor,
                      zeros_f16: torch.Tensor | None, *, group_size: int, sym: bool,
                      Y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y [m, d_out] fp32 = X [m, d_in] bf16 times the dequantized 4-bit weights (gptq_pack's
    qweight, scales_f16, zeros_f16) transposed."""
    if X.dtype != torch.bfloat16 or X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be a row-major bf16 [m, d_in] matrix")
    m, d_in = X.shape
    d_out = qweight.shape[0]
    if Y is None:
        Y = _empty(stream, (m, d_out), dtype=torch.float32, device=X.device)
    _check(lib().gptq_w4a16_matmul(_ptr(X), m, X.stride(0), _ptr(qweight), _ptr(scales_f16),
                                   _ptr(zeros_f16), d_out, d_in, group_size, int(bool(sym)),
                                   _ptr(Y), _stream(stream)), "gptq_w4a16_matmul")
    return Y


# -------------------------------------------------- running a quantized layer
# These calls take microseconds on the GPU, so the checks below are written to
# cost little: one condition on the way through, and the words only on the way
# out.  Devices are compared as indices (-1 for the host).
_W16_TYPES = (torch.int16, torch.uint16, torch.float16)
_W32_TYPES = (torch.int32, torch.uint32)
_FLOATS = (torch.bfloat16, torch.float32)


def _raw_stream(where: str, index: int, stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)  # current_stream() without its object
    if stream.device.index != index:
        raise ValueError(f"{where}: the stream is on {stream.device}, the tensors on GPU {index}")
    return stream.cuda_stream


def _call(where: str, index: int, f, *args):
    """The library call with the tensors' device as the current one."""
    if index == torch._C._cuda_getDevice():
        st = f(*args)
    else:
        with torch.cuda.device(index):
            st = f(*args)
    if st:
        raise GPTQError(st, where)


def _index(where: str, X: torch.Tensor, dtypes) -> int:
    """The GPU that the matrix X is on."""
    if X.dim() != 2 or X.dtype not in dtypes or not X.is_cuda:
        raise ValueError(f"{where}: X must be a GPU matrix of {dtypes}, got {X.dim()}-D "
                         f"{X.dtype} on {X.device}")
    return X.get_device()


def _rows(where: str, name: str, t: torch.Tensor, shape, dtypes, index: int) -> int:
    """Checks a row-major matrix and returns its leading dimension."""
    if not (t.shape == shape and t.dtype in dtypes and t.get_device() == index
            and (t.stride(1) == 1 or shape[1] == 1)):
        raise ValueError(f"{where}: {name} must be row-major {list(shape)} of {dtypes} on GPU "
                         f"{index}, got {list(t.shape)} {t.dtype} of strides {t.stride()} on "
                         f"{t.device}")
    return t.stride(0) if shape[0] > 1 else shape[1]


def _flat(where: str, name: str, t: torch.Tensor, shape, dtypes, index: int):
    if not (t.shape == shape and t.dtype in dtypes and t.get_device() == index
            and t.is_contiguous()):
        raise ValueError(f"{where}: {name} must be contiguous {list(shape)} of {dtypes} on GPU "
                         f"{index}, got {list(t.shape)} {t.dtype} of strides {t.stride()} on "
                         f"{t.device}")


def _scratch(where: str, ws, nbytes: int, X: torch.Tensor, stream):
    """The caller's workspace, or one of the call's own where it needs any."""
    if ws is None:
        return _workspace(nbytes, X.device, stream) if nbytes else None
    if ws.device != X.device or not ws.is_contiguous():
        raise ValueError(f"{where}: ws must be contiguous on {X.device}")
    return ws


def _span(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


def _w4_checks(where, X, x_dtype, qweight, scales_f16, zeros_f16, group_size, sym, Y, stream):
    """The packed weights' shapes against X's; returns (index, m, d_in, d_out, ldx, Y).  A group
    size that the library refuses is left to it: it reads nothing then."""
    index = _index(where, X, (x_dtype,))
    m, d_in = X.shape
    d_out = qweight.shape[0]
    if group_size == -1:
        meta = (d_out, 1)
    elif group_size > 0 and d_in % group_size == 0:
        meta = (d_out, d_in // group_size)
    else:
        meta = scales_f16.shape
    ldx, one = X.stride()
    if not (qweight.shape == (d_out, d_in // 8) and qweight.dtype in _W32_TYPES
            and qweight.is_contiguous() and qweight.get_device() == index
            and scales_f16.shape == meta and scales_f16.dtype in _W16_TYPES
            and scales_f16.is_contiguous() and scales_f16.get_device() == index
            and (sym or (zeros_f16 is not None and zeros_f16.shape == meta
                         and zeros_f16.dtype in _W16_TYPES and zeros_f16.is_contiguous()
                         and zeros_f16.get_device() == index))
            and (one == 1 or d_in == 1)):
        _flat(where, "qweight", qweight, (d_out, d_in // 8), _W32_TYPES, index)
        _flat(where, "scales_f16", scales_f16, meta, _W16_TYPES, index)
        if not sym:
            if zeros_f16 is None:
                raise ValueError(f"{where}: zeros_f16 is needed unless sym")
            _flat(where, "zeros_f16", zeros_f16, meta, _W16_TYPES, index)
        raise ValueError(f"{where}: X must be row-major, got strides {X.stride()}")
    if Y is None:
        Y = _empty(stream, (m, d_out), dtype=torch.float32, device=X.device)
    elif not (Y.shape == (m, d_out) and Y.dtype is torch.float32 and Y.is_contiguous()
              and Y.get_device() == index):
        _flat(where, "Y", Y, (m, d_out), (torch.float32,), index)
    return index, m, d_in, d_out, ldx if m > 1 else d_in, Y


@functools.lru_cache(maxsize=1024)
def gptq_w4a16_matvec_workspace(m: int, d_out: int, d_in: int, group_size: int) -> int:
    return int(lib().gptq_w4a16_matvec_workspace(m, d_out, d_in, group_size))


def gptq_w4a16_matvec(X: torch.Tensor, qweight: torch.Tensor, scales_f16: torch.Tensor,
                      zeros_f16: torch.Tensor | None, *, group_size: int, sym: bool,
                      Y: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """gptq_w4a16_matmul for the rows of a few tokens (m <= GPTQ_MATVEC_MAX_M), any d_in that is a
    multiple of 32: Y [m, d_out] fp32 = X [m, d_in] bf16 times the dequantized weights transposed."""
    where = "gptq_w4a16_matvec"
    index, m, d_in, d_out, ldx, Y = _w4_checks(where, X, torch.bfloat16, qweight, scales_f16,
                                               zeros_f16, group_size, sym, Y, stream)
    ws = _scratch(where, ws, gptq_w4a16_matvec_workspace(m, d_out, d_in, group_size), X, stream)
    _call(where, index, lib().gptq_w4a16_matvec, X.data_ptr(), m, ldx, qweight.data_ptr(),
          scales_f16.data_ptr(), None if sym else zeros_f16.data_ptr(), d_out, d_in, group_size,
          1 if sym else 0, Y.data_ptr(), *_span(ws), _raw_stream(where, index, stream))
    return Y


@functools.lru_cache(maxsize=1024)
def gptq_w4a8_workspace(m: int, d_out: int, d_in: int, group_size: int) -> int:
    return int(lib().gptq_w4a8_workspace(m, d_out, d_in, group_size))


def gptq_w4a8_matmul(X: torch.Tensor, x_scales: torch.Tensor, qweight: torch.Tensor,
                     scales_f16: torch.Tensor, zeros_f16: torch.Tensor | None, *,
                     group_size: int, sym: bool, Y: torch.Tensor | None = None,
                     ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y [m, d_out] fp32 = x_scales [m] times X [m, d_in] int8 (gptq_add_rmsnorm's 8-bit output)
    times the dequantized 4-bit weights transposed."""
    where = "gptq_w4a8_matmul"
    index, m, d_in, d_out, ldx, Y = _w4_checks(where, X, torch.int8, qweight, scales_f16,
                                               zeros_f16, group_size, sym, Y, stream)
    if not (x_scales.shape == (m,) and x_scales.dtype is torch.float32
            and x_scales.is_contiguous() and x_scales.get_device() == index):
        _flat(where, "x_scales", x_scales, (m,), (torch.float32,), index)
    ws = _scratch(where, ws, gptq_w4a8_workspace(m, d_out, d_in, group_size), X, stream)
    _call(where, index, lib().gptq_w4a8_matmul, X.data_ptr(), x_scales.data_ptr(), m, ldx,
          qweight.data_ptr(), scales_f16.data_ptr(), None if sym else zeros_f16.data_ptr(), d_out,
          d_in, group_size, 1 if sym else 0, Y.data_ptr(), *_span(ws),
          _raw_stream(where, index, stream))
    return Y


def gptq_add_rmsnorm(X: torch.Tensor, weight: torch.Tensor, *,
                     residual: torch.Tensor | None = None,
                     residual_out: torch.Tensor | None = None, eps: float = 1e-6,
                     out_dtype: torch.dtype = torch.int8, out: torch.Tensor | None = None,
                     out_scales: torch.Tensor | None = None, stream=None):
    """h = X + residual (X alone without one), then h weight / sqrt(mean h^2 + eps) per row, in
    bf16 or as int8 codes with an fp32 scale per row.  Returns (out, out_scales or None,
    residual_out or None); residual_out = residual updates the residual in place."""
    where = "gptq_add_rmsnorm"
    index = _index(where, X, _FLOATS)
    shape = X.shape
    m, d = shape
    if out_dtype is not torch.int8 and out_dtype is not torch.bfloat16:
        raise ValueError(f"{where}: out_dtype must be torch.int8 or torch.bfloat16")
    i8 = out_dtype is torch.int8
    if d > 1 and X.stride(1) != 1:
        raise ValueError(f"{where}: X must be row-major")
    _flat(where, "weight", weight, (d,), _FLOATS, index)
    r_code = ldr = ldro = r_ptr = ro_ptr = 0
    if residual is not None:
        ldr = _rows(where, "residual", residual, shape, _FLOATS, index)
        r_code = _dtype_code(residual)
        if residual_out is None:
            residual_out = _empty(stream, (m, d), dtype=residual.dtype, device=X.device)
        ldro = _rows(where, "residual_out", residual_out, shape, (residual.dtype,), index)
        r_ptr, ro_ptr = residual.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError(f"{where}: residual_out without residual")
    if out is None:
        out = _empty(stream, (m, d), dtype=out_dtype, device=X.device)
    ldo = _rows(where, "out", out, shape, (out_dtype,), index)
    if not i8:
        out_scales = None
    elif out_scales is None:
        out_scales = _empty(stream, m, dtype=torch.float32, device=X.device)
    else:
        _flat(where, "out_scales", out_scales, (m,), (torch.float32,), index)
    _call(where, index, lib().gptq_add_rmsnorm, X.data_ptr(), _dtype_code(X),
          X.stride(0) if m > 1 else d, r_ptr, r_code, ldr, ro_ptr, ldro, weight.data_ptr(),
          _dtype_code(weight), float(eps), m, d, out.data_ptr(), GPTQ_I8 if i8 else GPTQ_BF16, ldo,
          out_scales.data_ptr() if i8 else None, _raw_stream(where, index, stream))
    return out, out_scales, residual_out
