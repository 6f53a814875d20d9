"""Python binding of the 4-bit KV cache (``include/atom_kv4.h``): appending keys and values to its pages,
reading them back, and causal attention over it.

* ``kv4_cache(pages, page, heads, dim, device)``   -> ``KV4Cache`` (k, k_par, v, v_par)
* ``atom_kv4_append(K, V, slots, cache)``          writes the tokens' codes, zero points and scales
* ``atom_kv4_read(cache, slots, dtype)``           -> (K, V), what the codes in those slots stand for
* ``atom_kv4_attention(Q, cache, table, lens, q_start)`` -> out, as Q
* ``atom_kv4_attention_workspace_bytes(...)``

Argument marshalling only, as in the package's ``__init__``: shapes, types and devices are checked
before the call, a mismatch raises ``AtomError``.  Lengths, tables and slots stay on the device: a
call never synchronizes, and captures into a graph.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import bit_quantized_gemm_amd as _bq

from .w8a8 import check_device, check_rows, empty, fast_device, float_type, on_device

__all__ = ["KV4Cache", "kv4_cache", "atom_kv4_append", "atom_kv4_read", "atom_kv4_attention",
           "atom_kv4_attention_workspace_bytes"]

# Every symbol declared in include/atom_kv4.h.
EXPORTS = ("atom_kv4_append", "atom_kv4_read", "atom_kv4_attention_workspace_bytes", "atom_kv4_attention")


class _CCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("k_par", ctypes.c_void_p), ("v", ctypes.c_void_p), ("v_par", ctypes.c_void_p),
                ("pages", ctypes.c_int32), ("page", ctypes.c_int32), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32)]


class KV4Cache(NamedTuple):
    """The cache's arrays; any four tensors of these shapes will do wherever a cache is taken, as long as the zero points are
    whole numbers from 0 to 15 and the scales finite and not negative where sequences lie, as the append writes them."""
    k: object        # uint8 [pages, heads, page, dim / 2]
    k_par: object    # fp16  [pages, heads, page, 2]: (zero point, scale)
    v: object        # uint8 [pages, heads, page / 4, dim / 4, 8]
    v_par: object    # fp16  [pages, heads, page, 2]


def signatures():
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    pc = ctypes.POINTER(_CCache)
    return {
        "atom_kv4_append": (ctypes.c_int, [vp, i64, vp, i64, vp, i32, i32, pc, vp]),
        "atom_kv4_read": (ctypes.c_int, [pc, vp, i32, i32, vp, vp, vp]),
        "atom_kv4_attention_workspace_bytes": (i64, [i32] * 7),
        "atom_kv4_attention": (ctypes.c_int, [vp, i64, pc, vp, i32, vp, vp, i32, i32, i32, i32, i32, f32, i32, vp, vp,
                                              i64, vp]),
    }


def kv4_cache(pages, page, heads, dim, device="cuda"):
    """An empty cache: `pages` pages of `page` tokens for `heads` kv heads of `dim` channels, zeroed."""
    torch = _bq._torch()
    u8, f16 = torch.uint8, torch.float16
    return KV4Cache(torch.zeros((pages, heads, page, dim // 2), dtype=u8, device=device),
                    torch.zeros((pages, heads, page, 2), dtype=f16, device=device),
                    torch.zeros((pages, heads, page // 4, dim // 4, 8), dtype=u8, device=device),
                    torch.zeros((pages, heads, page, 2), dtype=f16, device=device))


def _sizes(cache):
    """(heads, dim) of a cache whose k has a valid shape."""
    try:
        k, _, _, _ = cache
    except (TypeError, ValueError):
        raise _bq.AtomError("cache must be four tensors (k, k_par, v, v_par)") from None
    if getattr(k, "dim", lambda: -1)() != 4:
        raise _bq.AtomError("the cache's k must be a 4-D tensor")
    pages, heads, page, half = k.shape
    if half not in (32, 64, 128) or page not in (16, 32, 64, 128, 256) or not 1 <= heads <= 1024 or pages < 1:
        raise _bq.AtomError(f"the cache's k has shape {tuple(k.shape)}, expected [pages, heads up to 1024, page 16 to "
                            "256, dim / 2 of 32, 64 or 128]")
    return heads, 2 * half


def _cache(cache, more=()):
    """(C struct, pointers of `more`) of a cache and the call's other contiguous tensors, all checked."""
    torch = _bq._torch()
    k, k_par, v, v_par = cache
    pages, heads, page, half = k.shape
    par = (pages, heads, page, 2)
    p = _bq._ptrs((k, "k", torch.uint8, None), (k_par, "k_par", torch.float16, par),
                  (v, "v", torch.uint8, (pages, heads, page // 4, half // 2, 8)), (v_par, "v_par", torch.float16, par),
                  *more)
    return _CCache(p[0], p[1], p[2], p[3], pages, page, heads, 2 * half), p[4:]


def _fast_cache(cache, d):
    """The C struct of a cache of well-formed tensors on device d, else None."""
    torch = _bq._torch()
    try:
        k, k_par, v, v_par = cache
        pages, heads, page, half = k.shape
        par, u8, f16 = (pages, heads, page, 2), torch.uint8, torch.float16
        if (half in (32, 64, 128) and page in (16, 32, 64, 128, 256) and 1 <= heads <= 1024 and pages
                and k.dtype is u8 and v.dtype is u8 and k_par.dtype is f16 and v_par.dtype is f16
                and v.shape == (pages, heads, page >> 2, half >> 1, 8) and k_par.shape == par and v_par.shape == par
                and k.is_contiguous() and k_par.is_contiguous() and v.is_contiguous() and v_par.is_contiguous()
                and k.get_device() == d and k_par.get_device() == d and v.get_device() == d and v_par.get_device() == d):
            return _CCache(k.data_ptr(), k_par.data_ptr(), v.data_ptr(), v_par.data_ptr(), pages, page, heads, 2 * half)
    except (AttributeError, TypeError, ValueError):
        pass
    return None


def _fast_rows(t, heads, dim, dtype, d):
    """The row distance of well-formed [tokens, heads, dim] rows on device d, else 0."""
    s = t.stride()
    inner = heads * dim
    if (t.dtype is dtype and s[2] == 1 and (s[1] == dim or heads == 1) and t.get_device() == d
            and (s[0] >= inner or t.shape[0] == 1)):
        return s[0] if t.shape[0] > 1 else inner
    return 0


def _same_device(t, name, cache):
    check_device(t, name)
    if t.get_device() != cache[0].get_device():
        raise _bq.AtomError(f"{name} is on {t.device}, the cache on {cache[0].device}")


def _tokens(slots):
    if getattr(slots, "dim", lambda: -1)() != 1:
        raise _bq.AtomError("slots must be a 1-D int64 tensor")
    return int(slots.shape[0])


def atom_kv4_append(K, V, slots, cache, stream=None):
    """Quantize K, V (fp16 / bf16 [tokens, heads, dim]; rows of heads * dim contiguous elements, which may lie
    apart) into the cache's slots (int64 [tokens]: page * page size + place; one outside the cache, such as
    -1, skips its token).  Two tokens of one call must not share a slot."""
    torch = _bq._torch()
    T = torch.Tensor
    if stream is None and type(K) is T and type(V) is T and type(slots) is T and K.is_cuda and K.dim() == 3:
        d, t = fast_device(K), K.dtype
        c = _fast_cache(cache, d) if d >= 0 and (t is torch.float16 or t is torch.bfloat16) else None
        if (c is not None and slots.dim() == 1 and K.shape == V.shape == (slots.shape[0], c.heads, c.dim)
                and slots.dtype is torch.int64 and slots.is_contiguous() and slots.get_device() == d):
            ks, vs = _fast_rows(K, c.heads, c.dim, t, d), _fast_rows(V, c.heads, c.dim, t, d)
            if ks and vs:
                status = _bq.load_library().atom_kv4_append(K.data_ptr(), ks, V.data_ptr(), vs, slots.data_ptr(), K.shape[0],
                                                            int(t is torch.bfloat16), c,
                                                            torch._C._cuda_getCurrentRawStream(d))
                if status:
                    _bq._check(status, "atom_kv4_append")
                return
    n = _tokens(slots)
    kind = float_type(K, "K")
    if float_type(V, "V") != kind:
        raise _bq.AtomError(f"V must be {K.dtype} (got {V.dtype})")
    shape = (n, *_sizes(cache))
    ks, vs = check_rows(K, "K", shape), check_rows(V, "V", shape)
    c, (pS,) = _cache(cache, ((slots, "slots", torch.int64, (n,)),))
    _same_device(K, "K", cache)
    _same_device(V, "V", cache)
    with on_device(K):
        _bq._check(_bq.load_library().atom_kv4_append(K.data_ptr(), ks, V.data_ptr(), vs, pS, n, kind, c,
                                                      _bq._stream(stream, K.device)), "atom_kv4_append")


def atom_kv4_read(cache, slots, dtype=None, K=None, V=None, stream=None):
    """(K, V) [tokens, heads, dim] that the codes in `slots` stand for, in `dtype` (default fp16, or K's);
    zeros for a slot outside the cache."""
    torch = _bq._torch()
    if stream is None and K is None and V is None and type(slots) is torch.Tensor and slots.is_cuda:
        d = fast_device(slots)
        t = torch.float16 if dtype is None else dtype
        c = _fast_cache(cache, d) if d >= 0 and (t is torch.float16 or t is torch.bfloat16) else None
        if c is not None and slots.dtype is torch.int64 and slots.dim() == 1 and slots.is_contiguous():
            n, device = slots.shape[0], slots.device
            K = torch.empty((n, c.heads, c.dim), dtype=t, device=device)
            V = torch.empty((n, c.heads, c.dim), dtype=t, device=device)
            status = _bq.load_library().atom_kv4_read(c, slots.data_ptr(), n, int(t is torch.bfloat16), K.data_ptr(),
                                                      V.data_ptr(), torch._C._cuda_getCurrentRawStream(d))
            if status:
                _bq._check(status, "atom_kv4_read")
            return K, V
    n = _tokens(slots)
    if dtype is None:
        dtype = K.dtype if K is not None else torch.float16
    if dtype not in (torch.float16, torch.bfloat16):
        raise _bq.AtomError(f"dtype must be torch.float16 or torch.bfloat16 (got {dtype})")
    heads, dim = _sizes(cache)
    K = empty((n, heads, dim), dtype, slots, stream) if K is None else K
    V = empty((n, heads, dim), dtype, slots, stream) if V is None else V
    c, (pS, pK, pV) = _cache(cache, ((slots, "slots", torch.int64, (n,)), (K, "K", dtype, (n, heads, dim)),
                                     (V, "V", dtype, (n, heads, dim))))
    with on_device(slots):
        _bq._check(_bq.load_library().atom_kv4_read(c, pS, n, int(dtype is torch.bfloat16), pK, pV,
                                                    _bq._stream(stream, slots.device)), "atom_kv4_read")
    return K, V


def atom_kv4_attention_workspace_bytes(total_q: int, q_heads: int, heads: int, dim: int, batch: int, max_q: int,
                                       max_len: int) -> int:
    r = _bq.load_library().atom_kv4_attention_workspace_bytes(total_q, q_heads, heads, dim, batch, max_q, max_len)
    if r < 0:
        raise _bq.AtomError(f"atom_kv4_attention_workspace_bytes: {_bq.atom_strerror(-r)}")
    return r


_attention_bytes = functools.lru_cache(maxsize=1024)(atom_kv4_attention_workspace_bytes)


def atom_kv4_attention(Q, cache, table, lens, q_start, scale=None, max_len=None, max_q=None, out=None, workspace=None,
                       stream=None):
    """Causal attention of each sequence's last tokens over its pages of the cache.

    Q (fp16 / bf16 [total_q, q_heads, dim]; rows may lie apart) holds the queries of sequence b in rows
    q_start[b] .. q_start[b + 1] - 1 (int32 [batch + 1]); they are the last of its lens[b] (int32 [batch]) tokens,
    which lie in the pages table[b] (int32 [batch, width]).  Query i of n sees tokens 0 .. lens[b] - n + i;
    one that sees none gets zeros, rows outside every sequence are left as they were.  `scale` defaults
    to dim ** -0.5.  `max_len` and `max_q` bound the lengths and query counts on the host (by default what
    the table and Q can hold; tighter bounds choose a better launch): queries behind max_q are left out, a length
    above max_len is taken as max_len.  `workspace`: 1-D uint8 of ``atom_kv4_attention_workspace_bytes`` bytes (calls that may overlap
    need one each), else a torch buffer is taken for the call when one is needed."""
    torch = _bq._torch()
    T = torch.Tensor
    if (stream is None and type(Q) is T and type(table) is T and type(lens) is T and type(q_start) is T and Q.is_cuda
            and Q.dim() == 3 and table.dim() == 2):
        d, t = fast_device(Q), Q.dtype
        c = _fast_cache(cache, d) if d >= 0 and (t is torch.float16 or t is torch.bfloat16) else None
        total, q_heads, dim = Q.shape
        batch, width = table.shape
        i32 = torch.int32
        if (c is not None and total and dim == c.dim and q_heads >= c.heads and q_heads % c.heads == 0
                and table.dtype is i32 and lens.dtype is i32 and q_start.dtype is i32 and batch and width
                and lens.shape == (batch,) and q_start.shape == (batch + 1,) and table.is_contiguous()
                and lens.is_contiguous() and q_start.is_contiguous() and table.get_device() == d
                and lens.get_device() == d and q_start.get_device() == d
                and (out is None or type(out) is T and out.dtype is t and out.shape == Q.shape and out.is_contiguous()
                     and out.get_device() == d)
                and (workspace is None or type(workspace) is T and workspace.dtype is torch.uint8
                     and workspace.dim() == 1 and workspace.is_contiguous() and workspace.get_device() == d)):
            qs = _fast_rows(Q, q_heads, dim, t, d)
            if qs:
                capacity = width * c.page
                max_len = capacity if max_len is None else max(1, min(int(max_len), capacity))
                max_q = total if max_q is None else max(1, min(int(max_q), total))
                if out is None:
                    out = torch.empty((total, q_heads, dim), dtype=t, device=Q.device)
                if workspace is None:
                    have = _attention_bytes(total, q_heads, c.heads, dim, batch, max_q, max_len)
                    if have:
                        workspace = torch.empty(have, dtype=torch.uint8, device=Q.device)
                else:
                    have = workspace.numel()
                status = _bq.load_library().atom_kv4_attention(
                    Q.data_ptr(), qs, c, table.data_ptr(), width, lens.data_ptr(), q_start.data_ptr(), total, q_heads,
                    batch, max_q, max_len, dim ** -0.5 if scale is None else float(scale), int(t is torch.bfloat16),
                    out.data_ptr(), None if workspace is None else workspace.data_ptr(), have,
                    torch._C._cuda_getCurrentRawStream(d))
                if status:
                    _bq._check(status, "atom_kv4_attention")
                return out
    if getattr(Q, "dim", lambda: -1)() != 3:
        raise _bq.AtomError("Q must be a 3-D tensor")
    kind = float_type(Q, "Q")
    total, q_heads, dim = Q.shape
    batch, width = _bq._mat(table, "table")
    if out is None:
        out = empty((total, q_heads, dim), Q.dtype, Q, stream)
    if workspace is not None and getattr(workspace, "dim", lambda: -1)() != 1:
        raise _bq.AtomError("workspace must be a 1-D uint8 tensor")
    heads, d = _sizes(cache)
    if dim != d:
        raise _bq.AtomError(f"Q has shape {tuple(Q.shape)}, expected a last dimension of {d}")
    if q_heads < heads or q_heads % heads:
        raise _bq.AtomError(f"Q has {q_heads} heads, no multiple of the cache's {heads} (shape {tuple(Q.shape)})")
    qs = check_rows(Q, "Q", Q.shape)
    c, p = _cache(cache, ((table, "table", torch.int32, (batch, width)), (lens, "lens", torch.int32, (batch,)),
                          (q_start, "q_start", torch.int32, (batch + 1,)), (out, "out", Q.dtype, (total, q_heads, dim)),
                          (workspace, "workspace", torch.uint8, None)))
    _same_device(Q, "Q", cache)
    capacity = width * c.page
    max_len = capacity if max_len is None else max(1, min(int(max_len), capacity))
    max_q = total if max_q is None else max(1, min(int(max_q), total))
    scale = dim ** -0.5 if scale is None else float(scale)
    pW, have = p[4], 0
    if workspace is None:
        have = _attention_bytes(total, q_heads, heads, dim, batch, max_q, max_len)
        if have:
            workspace = empty((have,), torch.uint8, Q, stream)
            pW = workspace.data_ptr()
    else:
        have = int(workspace.numel())
    with on_device(Q):
        _bq._check(_bq.load_library().atom_kv4_attention(Q.data_ptr(), qs, c, p[0], width, p[1], p[2], total, q_heads,
                                                         batch, max_q, max_len, scale, kind, p[3], pW, have,
                                                         _bq._stream(stream, Q.device)), "atom_kv4_attention")
    return out
