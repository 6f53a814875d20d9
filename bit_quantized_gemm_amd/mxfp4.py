"""Python binding of the MXFP4 linear layer (``include/atom_mxfp4.h``): microscaled 4-bit floating point on both sides
(E2M1 codes, one E8M0 scale for each 32 values), fp16 or bf16 in and out.

* ``atom_quantize_mxfp4(X)``                   -> (Xq uint8 [rows, row bytes], sx uint8 [groups, rows, 8]); weights too (offline)
* ``atom_dequantize_mxfp4(Xq, sx, K)``         -> X [rows, K], what the codes stand for
* ``atom_gemm_mxfp4(Xq, sx, Wq, sw, K)``       -> Y [M, N]
* ``linear_mxfp4(X, Wq, sw, bias)``            -> Y [M, N]: both in one call
* ``atom_mxfp4_row_bytes(K)``, ``atom_mxfp4_groups(K)``, ``atom_gemm_mxfp4_workspace_bytes(M, N, K)``,
  ``atom_linear_mxfp4_workspace_bytes(M, N, K)``

Argument marshalling only, as in the package's ``__init__``: shapes, types and devices are checked
before the call, a mismatch raises ``AtomError``.
"""
from __future__ import annotations

import ctypes
import functools

import bit_quantized_gemm_amd as _bq

from .w8a8 import _bytes, check_device, check_rows, empty, float_type, on_device

__all__ = ["atom_mxfp4_row_bytes", "atom_mxfp4_groups", "atom_quantize_mxfp4", "atom_dequantize_mxfp4",
           "atom_gemm_mxfp4_workspace_bytes", "atom_gemm_mxfp4", "atom_linear_mxfp4_workspace_bytes", "linear_mxfp4"]

# Every symbol declared in include/atom_mxfp4.h.
EXPORTS = ("atom_mxfp4_row_bytes", "atom_mxfp4_groups", "atom_quantize_mxfp4", "atom_dequantize_mxfp4",
           "atom_gemm_mxfp4_workspace_bytes", "atom_gemm_mxfp4", "atom_linear_mxfp4_workspace_bytes", "atom_linear_mxfp4")


def signatures():
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    return {
        "atom_mxfp4_row_bytes": (i64, [i32]),
        "atom_mxfp4_groups": (i32, [i32]),
        "atom_quantize_mxfp4": (ctypes.c_int, [vp, i64, i32, i32, i32, vp, vp, vp]),
        "atom_dequantize_mxfp4": (ctypes.c_int, [vp, vp, i32, i32, i32, vp, vp]),
        "atom_gemm_mxfp4_workspace_bytes": (i64, [i32, i32, i32]),
        "atom_gemm_mxfp4": (ctypes.c_int, [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, i64, vp]),
        "atom_linear_mxfp4_workspace_bytes": (i64, [i32, i32, i32]),
        "atom_linear_mxfp4": (ctypes.c_int, [vp, i64, i32, vp, vp, vp, i32, i32, i32, vp, vp, i64, vp]),
    }


def atom_mxfp4_row_bytes(K: int) -> int:
    return int(_bq.load_library().atom_mxfp4_row_bytes(_bq._c_int(K)))


def atom_mxfp4_groups(K: int) -> int:
    return int(_bq.load_library().atom_mxfp4_groups(_bq._c_int(K)))


@functools.lru_cache(maxsize=256)
def packed(K):
    """(row bytes, groups) of a valid K, else AtomError."""
    r = atom_mxfp4_row_bytes(K)
    if r < 0:
        _bq._check(-r, f"K={K}")
    return r, atom_mxfp4_groups(K)


def atom_gemm_mxfp4_workspace_bytes(M: int, N: int, K: int) -> int:
    return _bytes("atom_gemm_mxfp4_workspace_bytes", M, N, K)


def atom_linear_mxfp4_workspace_bytes(M: int, N: int, K: int) -> int:
    return _bytes("atom_linear_mxfp4_workspace_bytes", M, N, K)


_linear_bytes = functools.lru_cache(maxsize=1024)(atom_linear_mxfp4_workspace_bytes)


def atom_quantize_mxfp4(X, Xq=None, sx=None, stream=None):
    """Codes and scales of the rows of X (fp16 / bf16 [rows, K]; rows may lie apart)."""
    if stream is None and Xq is None and sx is None and _bq._SHORT is not None:
        out = _bq._SHORT.quantize_mxfp4(X)
        if out is not None:
            return out
    torch = _bq._torch()
    u8 = torch.uint8
    rows, K = _bq._mat(X, "X")
    kind = float_type(X, "X")
    rb, g = packed(K)
    ldx = check_rows(X, "X", (rows, K))
    if Xq is None:
        Xq = empty((rows, rb), u8, X, stream)
    if sx is None:
        sx = empty((g, rows, 8), u8, X, stream)
    pQ, pS = _bq._ptrs((Xq, "Xq", u8, (rows, rb)), (sx, "sx", u8, (g, rows, 8)))
    check_device(X, "X")
    if X.get_device() != Xq.get_device():
        raise _bq.AtomError(f"Xq is on {Xq.device}, the other operands on {X.device}")
    with on_device(X):
        _bq._check(_bq.load_library().atom_quantize_mxfp4(X.data_ptr(), ldx, kind, rows, K, pQ, pS,
                                                          _bq._stream(stream, X.device)), "atom_quantize_mxfp4")
    return Xq, sx


def atom_dequantize_mxfp4(Xq, sx, K, dtype=None, X=None, stream=None):
    """X [rows, K] that packed rows stand for, in `dtype` (default fp16, or X's)."""
    torch = _bq._torch()
    u8 = torch.uint8
    if stream is None and X is None and _bq._SHORT is not None and dtype in (None, torch.float16, torch.bfloat16):
        X = _bq._SHORT.dequantize_mxfp4(Xq, sx, K, dtype is torch.bfloat16)
        if X is not None:
            return X
    K = int(K)
    rb, g = packed(K)
    rows, _ = _bq._mat(Xq, "Xq")
    dtype = dtype if dtype is not None else X.dtype if isinstance(X, torch.Tensor) else torch.float16
    if dtype not in (torch.float16, torch.bfloat16):
        raise _bq.AtomError(f"dtype must be torch.float16 or torch.bfloat16 (got {dtype})")
    if X is None:
        X = empty((rows, K), dtype, Xq, stream)
    pQ, pS, pX = _bq._ptrs((Xq, "Xq", u8, (rows, rb)), (sx, "sx", u8, (g, rows, 8)), (X, "X", dtype, (rows, K)))
    with on_device(Xq):
        _bq._check(_bq.load_library().atom_dequantize_mxfp4(pQ, pS, rows, K, int(dtype is torch.bfloat16), pX,
                                                            _bq._stream(stream, Xq.device)), "atom_dequantize_mxfp4")
    return X


def atom_gemm_mxfp4(Xq, sx, Wq, sw, K, bias=None, Y=None, dtype=None, workspace=None, stream=None):
    """Y [M, N] of packed operands; its type is Y's, or the bias's, or `dtype` (default fp16).  With a
    workspace (1-D uint8, ``atom_gemm_mxfp4_workspace_bytes``) grids of few output tiles divide K; without one, or with less, they
    take up to twice as long (``linear_mxfp4`` takes one for itself).  Calls that may overlap need one each."""
    torch = _bq._torch()
    if stream is None and Y is None and _bq._SHORT is not None:
        kind = dtype if dtype is not None else getattr(bias, "dtype", torch.float16)
        if kind is torch.float16 or kind is torch.bfloat16:
            Y = _bq._SHORT.gemm_mxfp4(Xq, sx, Wq, sw, K, bias, kind is torch.bfloat16, workspace)
            if Y is not None:
                return Y
    K = int(K)
    rb, g = packed(K)
    M, _ = _bq._mat(Xq, "Xq")
    N, _ = _bq._mat(Wq, "Wq")
    given = {t.dtype for t in (Y, bias) if isinstance(t, torch.Tensor)} | ({dtype} if dtype is not None else set())
    if len(given) > 1:
        raise _bq.AtomError(f"Y, bias and dtype must agree (got {sorted(map(str, given))})")
    dtype = given.pop() if given else torch.float16
    if dtype not in (torch.float16, torch.bfloat16):
        raise _bq.AtomError(f"Y must be torch.float16 or torch.bfloat16 (got {dtype})")
    if Y is None:
        Y = empty((M, N), dtype, Xq, stream)
    if workspace is not None and getattr(workspace, "dim", lambda: -1)() != 1:
        raise _bq.AtomError("workspace must be a 1-D uint8 tensor")
    u8 = torch.uint8
    p = _bq._ptrs((Xq, "Xq", u8, (M, rb)), (sx, "sx", u8, (g, M, 8)), (Wq, "Wq", u8, (N, rb)), (sw, "sw", u8, (g, N, 8)),
                  (bias, "bias", dtype, (N,)), (Y, "Y", dtype, (M, N)), (workspace, "workspace", u8, None))
    with on_device(Xq):
        _bq._check(_bq.load_library().atom_gemm_mxfp4(p[0], p[1], p[2], p[3], p[4], M, N, K, int(dtype is torch.bfloat16),
                                                      p[5], p[6], 0 if workspace is None else int(workspace.numel()),
                                                      _bq._stream(stream, Xq.device)), "atom_gemm_mxfp4")
    return Y


def linear_mxfp4(X, Wq, sw, bias=None, Y=None, workspace=None, stream=None):
    """The layer: X (fp16 / bf16 [M, K]; rows may lie apart) quantized and multiplied with packed weights in
    one call.  Y has X's type.  `workspace`: 1-D uint8 of at least ``atom_linear_mxfp4_workspace_bytes``
    bytes (calls that may overlap need one each; none for few tokens or outputs, which take one launch), else a torch buffer is
    taken for the call when one is needed."""
    if stream is None and Y is None and workspace is None and _bq._SHORT is not None:
        Y = _bq._SHORT.linear_mxfp4(X, Wq, sw, bias)
        if Y is not None:
            return Y
    torch = _bq._torch()
    u8 = torch.uint8
    M, K = _bq._mat(X, "X")
    N, _ = _bq._mat(Wq, "Wq")
    kind = float_type(X, "X")
    rb, g = packed(K)
    ldx = check_rows(X, "X", (M, K))
    need = _linear_bytes(M, N, K)
    if Y is None:
        Y = empty((M, N), X.dtype, X, stream)
    if workspace is None:
        workspace = empty((need,), u8, X, stream) if need else None
    elif getattr(workspace, "dim", lambda: -1)() != 1:
        raise _bq.AtomError("workspace must be a 1-D uint8 tensor")
    elif workspace.numel() < need:
        raise _bq.AtomError(f"workspace has shape {tuple(workspace.shape)}, expected at least ({need},)")
    p = _bq._ptrs((Y, "Y", X.dtype, (M, N)), (Wq, "Wq", u8, (N, rb)), (sw, "sw", u8, (g, N, 8)),
                  (bias, "bias", X.dtype, (N,)), (workspace, "workspace", u8, None))
    check_device(X, "X")
    if X.get_device() != Y.get_device():
        raise _bq.AtomError(f"X is on {X.device}, the other operands on {Y.device}")
    with on_device(X):
        _bq._check(_bq.load_library().atom_linear_mxfp4(X.data_ptr(), ldx, kind, p[1], p[2], p[3], M, N, K, p[0], p[4],
                                                        0 if workspace is None else int(workspace.numel()),
                                                        _bq._stream(stream, X.device)), "atom_linear_mxfp4")
    return Y
