"""Python binding of the W8A8 linear layer (``include/atom_w8a8.h``): int8 codes on both sides, one fp32
scale for each token and one for each output channel, fp16 or bf16 in and out.

* ``atom_quantize_w8a8(X)``                     -> (Xq int8 [rows, row bytes], sx fp32 [rows]); weights too (offline)
* ``atom_gemm_w8a8(Xq, sx, Wq, sw, K)``         -> Y [M, N]
* ``linear_w8a8(X, Wq, sw, bias)``              -> Y [M, N]: both in one call
* ``atom_w8a8_row_bytes(K)``, ``atom_gemm_w8a8_workspace_bytes(M, N, K)``,
  ``atom_linear_w8a8_workspace_bytes(M, N, K)``

Argument marshalling only, as in the package's ``__init__``: shapes, types and devices are checked
before the call, a mismatch raises ``AtomError``.
"""
from __future__ import annotations

import ctypes
import functools

import bit_quantized_gemm_amd as _bq

__all__ = ["atom_w8a8_row_bytes", "atom_quantize_w8a8", "atom_gemm_w8a8_workspace_bytes", "atom_gemm_w8a8",
           "atom_linear_w8a8_workspace_bytes", "linear_w8a8"]

# Every symbol declared in include/atom_w8a8.h.
EXPORTS = ("atom_w8a8_row_bytes", "atom_quantize_w8a8", "atom_gemm_w8a8_workspace_bytes", "atom_gemm_w8a8",
           "atom_linear_w8a8_workspace_bytes", "atom_linear_w8a8")


def signatures():
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    return {
        "atom_w8a8_row_bytes": (i64, [i32]),
        "atom_quantize_w8a8": (ctypes.c_int, [vp, i64, i32, i32, i32, vp, vp, vp]),
        "atom_gemm_w8a8_workspace_bytes": (i64, [i32, i32, i32]),
        "atom_gemm_w8a8": (ctypes.c_int, [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, i64, vp]),
        "atom_linear_w8a8_workspace_bytes": (i64, [i32, i32, i32]),
        "atom_linear_w8a8": (ctypes.c_int, [vp, i64, i32, vp, vp, vp, i32, i32, i32, vp, vp, i64, vp]),
    }


def float_type(t, name):
    """The C ABI's number of a 16-bit float tensor's type."""
    torch = _bq._torch()
    if not isinstance(t, torch.Tensor):
        raise _bq.AtomError(f"{name} must be a torch.Tensor")
    if t.dtype is torch.float16:
        return 0
    if t.dtype is torch.bfloat16:
        return 1
    raise _bq.AtomError(f"{name} must be torch.float16 or torch.bfloat16 (got {t.dtype})")


class on_device:
    """The tensor's device as the current one during a call: kernels are launched on the current device,
    and the stream belongs to the tensor's."""

    def __init__(self, t):
        torch = _bq._torch()
        i = t.get_device()
        self._guard = torch.cuda.device(i) if t.is_cuda and i != torch.cuda.current_device() else None

    def __enter__(self):
        if self._guard is not None:
            self._guard.__enter__()

    def __exit__(self, *a):
        if self._guard is not None:
            self._guard.__exit__(*a)


def empty(shape, dtype, like, stream):
    """A new tensor for a call on `stream` (None: the current one).  The allocator hands out memory in the order
    of one stream's work, so what a call on another stream writes has to be allocated there."""
    if stream is None:
        return _bq._empty(shape, dtype, like)
    with _bq._torch().cuda.stream(stream):
        return _bq._empty(shape, dtype, like)


def fast_device(t):
    """The device number of a tensor on the current device, else -1.  Calls on the current stream of the current
    device whose arguments all pass take the short way (8 us less of host time a call than the full checks, which name
    the first problem and serve every other call)."""
    d = t.get_device()
    return d if d == _bq._torch()._C._cuda_getDevice() else -1


def check_rows(t, name, shape):
    """A tensor of `shape` whose last dimensions are contiguous within a row: returns the distance of its
    rows in elements.  (Rows may lie apart, as in a slice of a wider projection.)"""
    if tuple(t.shape) != tuple(shape):
        raise _bq.AtomError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    inner = 1
    for n, s in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if n != 1 and s != inner:
            raise _bq.AtomError(f"{name} must be contiguous within a row")
        inner *= n
    if t.shape[0] > 1 and t.stride(0) < inner:
        raise _bq.AtomError(f"{name} must be contiguous within a row, and its rows may not overlap")
    return int(t.stride(0)) if t.shape[0] > 1 else inner


def check_device(t, name):
    if not t.is_cuda:
        raise _bq.AtomError(f"{name} must be a ROCm device tensor (got {t.device}); there is no CPU path")


def _bytes(what, M, N, K):
    r = getattr(_bq.load_library(), what)(M, N, K)
    if r < 0:
        raise _bq.AtomError(f"{what}: {_bq.atom_strerror(-r)}")
    return r


def atom_w8a8_row_bytes(K: int) -> int:
    return int(_bq.load_library().atom_w8a8_row_bytes(K))


@functools.lru_cache(maxsize=256)
def _row_bytes(K):
    r = atom_w8a8_row_bytes(K)
    if r < 0:
        _bq._check(-r, f"K={K}")
    return r


def atom_gemm_w8a8_workspace_bytes(M: int, N: int, K: int) -> int:
    return _bytes("atom_gemm_w8a8_workspace_bytes", M, N, K)


def atom_linear_w8a8_workspace_bytes(M: int, N: int, K: int) -> int:
    return _bytes("atom_linear_w8a8_workspace_bytes", M, N, K)


_linear_bytes = functools.lru_cache(maxsize=1024)(atom_linear_w8a8_workspace_bytes)


def atom_quantize_w8a8(X, Xq=None, sx=None, stream=None):
    """Codes and scales of the rows of X (fp16 / bf16 [rows, K]; rows may lie apart)."""
    torch = _bq._torch()
    rows, K = _bq._mat(X, "X")
    kind = float_type(X, "X")
    rb = _row_bytes(K)
    ldx = check_rows(X, "X", (rows, K))
    if Xq is None:
        Xq = empty((rows, rb), torch.int8, X, stream)
    if sx is None:
        sx = empty((rows,), torch.float32, X, stream)
    pQ, pS = _bq._ptrs((Xq, "Xq", torch.int8, (rows, rb)), (sx, "sx", torch.float32, (rows,)))
    check_device(X, "X")
    if X.get_device() != Xq.get_device():
        raise _bq.AtomError(f"Xq is on {Xq.device}, the other operands on {X.device}")
    with on_device(X):
        _bq._check(_bq.load_library().atom_quantize_w8a8(X.data_ptr(), ldx, kind, rows, K, pQ, pS,
                                                         _bq._stream(stream, X.device)), "atom_quantize_w8a8")
    return Xq, sx


def atom_gemm_w8a8(Xq, sx, Wq, sw, K, bias=None, Y=None, dtype=None, workspace=None, stream=None):
    """Y [M, N] of packed operands; its type is Y's, or the bias's, or `dtype` (default fp16).  With a
    workspace (1-D uint8, ``atom_gemm_w8a8_workspace_bytes``) grids of few output tiles divide K."""
    torch = _bq._torch()
    rb = _row_bytes(int(K))
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
    p = _bq._ptrs((Xq, "Xq", torch.int8, (M, rb)), (sx, "sx", torch.float32, (M,)), (Wq, "Wq", torch.int8, (N, rb)),
                  (sw, "sw", torch.float32, (N,)), (bias, "bias", dtype, (N,)), (Y, "Y", dtype, (M, N)),
                  (workspace, "workspace", torch.uint8, None))
    with on_device(Xq):
        _bq._check(_bq.load_library().atom_gemm_w8a8(p[0], p[1], p[2], p[3], p[4], M, N, K, int(dtype is torch.bfloat16),
                                                     p[5], p[6], 0 if workspace is None else int(workspace.numel()),
                                                     _bq._stream(stream, Xq.device)), "atom_gemm_w8a8")
    return Y


def linear_w8a8(X, Wq, sw, bias=None, Y=None, workspace=None, stream=None):
    """The layer: X (fp16 / bf16 [M, K]; rows may lie apart) quantized and multiplied with packed weights in
    one call.  Y has X's type.  `workspace`: 1-D uint8 of at least ``atom_linear_w8a8_workspace_bytes``
    bytes (calls that may overlap need one each; none for the few tokens that take one launch), else a torch buffer is
    taken for the call when one is needed."""
    torch = _bq._torch()
    T = torch.Tensor
    if stream is None and Y is None and workspace is None and type(X) is T and type(Wq) is T and type(sw) is T:
        t, xs, ws = X.dtype, X.shape, Wq.shape
        if X.is_cuda and len(xs) == 2 and len(ws) == 2 and (t is torch.float16 or t is torch.bfloat16):
            M, K = xs
            N = ws[0]
            ldx, step = X.stride()
            d = fast_device(X)
            if (d >= 0 and 1 <= K <= _bq.MAX_K and M and N and (step == 1 or K == 1) and (ldx >= K or M == 1)
                    and Wq.dtype is torch.int8 and ws[1] == (K + 127 & -128) and Wq.is_contiguous()
                    and Wq.get_device() == d and sw.dtype is torch.float32 and sw.shape == (N,) and sw.is_contiguous()
                    and sw.get_device() == d
                    and (bias is None or type(bias) is T and bias.dtype is t and bias.shape == (N,)
                         and bias.is_contiguous() and bias.get_device() == d)):
                need = _linear_bytes(M, N, K)
                Y = X.new_empty((M, N))
                workspace = torch.empty(need, dtype=torch.uint8, device=X.device) if need else None
                status = _bq.load_library().atom_linear_w8a8(
                    X.data_ptr(), ldx, int(t is torch.bfloat16), Wq.data_ptr(), sw.data_ptr(),
                    None if bias is None else bias.data_ptr(), M, N, K, Y.data_ptr(), workspace.data_ptr() if need else None, need,
                    torch._C._cuda_getCurrentRawStream(d))
                if status:
                    _bq._check(status, "atom_linear_w8a8")
                return Y
    M, K = _bq._mat(X, "X")
    N, _ = _bq._mat(Wq, "Wq")
    kind = float_type(X, "X")
    rb = _row_bytes(K)
    ldx = check_rows(X, "X", (M, K))
    need = _linear_bytes(M, N, K)
    if Y is None:
        Y = empty((M, N), X.dtype, X, stream)
    if workspace is None:
        workspace = empty((need,), torch.uint8, X, stream) if need else None
    elif getattr(workspace, "dim", lambda: -1)() != 1:
        raise _bq.AtomError("workspace must be a 1-D uint8 tensor")
    elif workspace.numel() < need:
        raise _bq.AtomError(f"workspace has shape {tuple(workspace.shape)}, expected at least ({need},)")
    p = _bq._ptrs((Y, "Y", X.dtype, (M, N)), (Wq, "Wq", torch.int8, (N, rb)), (sw, "sw", torch.float32, (N,)),
                  (bias, "bias", X.dtype, (N,)), (workspace, "workspace", torch.uint8, None))
    check_device(X, "X")
    if X.get_device() != Y.get_device():
        raise _bq.AtomError(f"X is on {X.device}, the other operands on {Y.device}")
    with on_device(X):
        _bq._check(_bq.load_library().atom_linear_w8a8(X.data_ptr(), ldx, kind, p[1], p[2], p[3], M, N, K, p[0], p[4],
                                                       0 if workspace is None else int(workspace.numel()), _bq._stream(stream, X.device)),
                   "atom_linear_w8a8")
    return Y
