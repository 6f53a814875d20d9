"""Python binding of the root-mean-square norm in front of the quantized layers (``include/atom_norm.h``): the residual's
addition, the norm and the rows' quantization in one pass.

* ``atom_rmsnorm_w8a8(X, weight, eps, residual)``   -> (Xq, sx, H): rows as ``atom_gemm_w8a8`` takes them
* ``atom_rmsnorm_mxfp4(X, weight, eps, residual)``  -> (Xq, sx, H): rows as ``atom_gemm_mxfp4`` takes them

H is the sum X + residual (None without a residual).  Argument marshalling only, as in the package's ``__init__``: shapes,
types and devices are checked before the call, a mismatch raises ``AtomError``.
"""
from __future__ import annotations

import ctypes

import bit_quantized_gemm_amd as _bq

from .mxfp4 import packed
from .w8a8 import _row_bytes, check_device, check_rows, empty, float_type, on_device

__all__ = ["atom_rmsnorm_w8a8", "atom_rmsnorm_mxfp4"]

# Every symbol declared in include/atom_norm.h.
EXPORTS = ("atom_rmsnorm_w8a8", "atom_rmsnorm_mxfp4")


def signatures():
    vp, i32, i64, f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double
    args = [vp, i64, vp, i64, vp, f64, i32, i32, i32, vp, i64, vp, vp, vp]
    return {name: (ctypes.c_int, args) for name in EXPORTS}


def _rmsnorm(name, mx, X, weight, eps, residual, H, Xq, sx, stream):
    if stream is None and H is None and Xq is None and sx is None and _bq._SHORT is not None:
        out = (_bq._SHORT.rmsnorm_mxfp4 if mx else _bq._SHORT.rmsnorm_w8a8)(X, weight, float(eps), residual)
        if out is not None:
            return out
    rows, K = _bq._mat(X, "X")
    kind = float_type(X, "X")
    (qs, qt), (ss, st) = (_mx if mx else _w8)(rows, K)
    ldx = check_rows(X, "X", (rows, K))
    if residual is None and H is not None:
        raise _bq.AtomError("H must be None without a residual")
    ldr = ldh = K
    if residual is not None:
        if float_type(residual, "residual") != kind:
            raise _bq.AtomError(f"residual must be {X.dtype} (got {residual.dtype})")
        ldr = check_rows(residual, "residual", (rows, K))
        if H is None:
            H = empty((rows, K), X.dtype, X, stream)
        elif float_type(H, "H") != kind:
            raise _bq.AtomError(f"H must be {X.dtype} (got {H.dtype})")
        ldh = check_rows(H, "H", (rows, K))
    Xq = empty(qs, qt, X, stream) if Xq is None else Xq
    sx = empty(ss, st, X, stream) if sx is None else sx
    pW, pQ, pS = _bq._ptrs((weight, "weight", X.dtype, (K,)), (Xq, "Xq", qt, qs), (sx, "sx", st, ss))
    for t, n in ((X, "X"), (residual, "residual"), (H, "H")):
        if t is not None:
            check_device(t, n)
            if t.get_device() != Xq.get_device():
                raise _bq.AtomError(f"{n} is on {t.device}, the other operands on {Xq.device}")
    with on_device(X):
        call = getattr(_bq.load_library(), name)
        _bq._check(call(X.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr, pW, float(eps), kind, rows, K,
                        None if H is None else H.data_ptr(), ldh, pQ, pS, _bq._stream(stream, X.device)), name)
    return Xq, sx, H


def _w8(rows, K):
    torch = _bq._torch()
    return ((rows, _row_bytes(K)), torch.int8), ((rows,), torch.float32)


def _mx(rows, K):
    rb, g = packed(K)
    u8 = _bq._torch().uint8
    return ((rows, rb), u8), ((g, rows, 8), u8)


def atom_rmsnorm_w8a8(X, weight, eps=1e-6, residual=None, H=None, Xq=None, sx=None, stream=None):
    """The rows of X (fp16 / bf16 [rows, K]; rows may lie apart), plus `residual` if one is given, normed and quantized to
    int8: (Xq int8 [rows, row bytes], sx fp32 [rows], H).  H, the sum in X's type, is what the next layer's residual is;
    it may be given as the residual (or X) itself, which is then replaced."""
    return _rmsnorm("atom_rmsnorm_w8a8", False, X, weight, eps, residual, H, Xq, sx, stream)


def atom_rmsnorm_mxfp4(X, weight, eps=1e-6, residual=None, H=None, Xq=None, sx=None, stream=None):
    """As ``atom_rmsnorm_w8a8``, quantized to MXFP4: (Xq uint8 [rows, row bytes], sx uint8 [groups, rows, 8], H)."""
    return _rmsnorm("atom_rmsnorm_mxfp4", True, X, weight, eps, residual, H, Xq, sx, stream)
