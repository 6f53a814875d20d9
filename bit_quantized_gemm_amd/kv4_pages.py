"""Python binding of the 4-bit KV cache's bookkeeping (``include/atom_kv4_pages.h``): block tables, slots and a pool of free
pages that live on the device.

* ``kv4_pool(pages, device)``                                   -> ``KV4Pool`` (free, state), every page free
* ``atom_kv4_extend(lens, new, table, pool, page, total)``      -> (slots, q_start, lens, state) of a step's new tokens
* ``atom_kv4_release(done, lens, table, pool, page)``           -> (lens, state) behind the sequences that are done

The results are what ``atom_kv4_append`` (slots) and ``atom_kv4_attention`` (table, lens, q_start) take.  Argument marshalling
only, as in the package's ``__init__``: shapes, types and devices are checked before the call, a mismatch raises ``AtomError``.
Nothing synchronizes, and calls capture into a graph.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import bit_quantized_gemm_amd as _bq

from .w8a8 import empty, on_device

__all__ = ["KV4Pool", "kv4_pool", "atom_kv4_extend", "atom_kv4_release"]

# Every symbol declared in include/atom_kv4_pages.h.
EXPORTS = ("atom_kv4_extend", "atom_kv4_release")


class KV4Pool(NamedTuple):
    """The pool's arrays; any two tensors of these shapes will do wherever a pool is taken."""
    free: object     # int32 [capacity]: the first state[0] are free pages, the next one to be taken last
    state: object    # int32 [2]: (free pages, pages that the last step was missing)


def signatures():
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    return {
        "atom_kv4_extend": (ctypes.c_int, [vp, vp, vp, i32, i32, i32, vp, i32, vp, vp, i32, vp, vp, vp, vp]),
        "atom_kv4_release": (ctypes.c_int, [vp, vp, vp, i32, i32, i32, vp, i32, vp, vp, vp, vp]),
    }


def kv4_pool(pages, device="cuda"):
    """A pool of the pages 0 .. pages - 1, all free; they are taken in this order."""
    torch = _bq._torch()
    return KV4Pool(torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=device),
                   torch.tensor([pages, 0], dtype=torch.int32, device=device))


def _pool(pool):
    try:
        free, state = pool
    except (TypeError, ValueError):
        raise _bq.AtomError("pool must be two tensors (free, state)") from None
    if getattr(free, "dim", lambda: -1)() != 1:
        raise _bq.AtomError("the pool's free must be a 1-D int32 tensor")
    return free, state


def atom_kv4_extend(lens, new, table, pool, page, total, slots=None, q_start=None, lens_out=None, state_out=None, stream=None):
    """Admit new[b] tokens (int32 [batch]) to each sequence of lens[b] (int32 [batch]): pages of `page` tokens are taken from the
    pool where none of the sequence's holds them yet, and written into its row of `table` (int32 [batch, width]).

    `total` is the number of rows that hold all new tokens, one sequence behind the other.  Returns (slots int64 [total]: each
    row's slot, -1 for rows behind the last one; q_start int32 [batch + 1]; lens_out int32 [batch], with the new tokens; state_out
    int32 [2]: the pool's new state).  The inputs stay as they were but for the table, unless lens_out is lens or state_out
    the pool's state, which are then replaced (more than 1024 rows take a second launch for it).  If the pool holds
    too few pages nothing is taken: all slots are -1, lengths and pool stay, state_out[1] says how many are missing."""
    free, state = _pool(pool)
    total, page = _bq._size(total, "total"), _bq._size(page, "page")
    if stream is None and slots is None and q_start is None and lens_out is None and state_out is None and _bq._SHORT is not None:
        out = _bq._SHORT.kv4_extend(lens, new, table, free, state, page, total)
        if out is not None:
            return out
    torch = _bq._torch()
    i32 = torch.int32
    batch, width = _bq._mat(table, "table")
    if total < 1:
        raise _bq.AtomError(f"total must be at least 1 (got {total})")
    slots = empty((total,), torch.int64, table, stream) if slots is None else slots
    q_start = empty((batch + 1,), i32, table, stream) if q_start is None else q_start
    lens_out = empty((batch,), i32, table, stream) if lens_out is None else lens_out
    state_out = empty((2,), i32, table, stream) if state_out is None else state_out
    p = _bq._ptrs((lens, "lens", i32, (batch,)), (new, "new", i32, (batch,)), (table, "table", i32, (batch, width)),
                  (free, "free", i32, None), (state, "state", i32, (2,)), (slots, "slots", torch.int64, (total,)),
                  (q_start, "q_start", i32, (batch + 1,)), (lens_out, "lens_out", i32, (batch,)),
                  (state_out, "state_out", i32, (2,)))
    with on_device(table):
        _bq._check(_bq.load_library().atom_kv4_extend(p[0], p[1], p[2], batch, width, page, p[3], _bq._c_int(free.shape[0]), p[4],
                                                      p[5], total, p[6], p[7], p[8], _bq._stream(stream, table.device)),
                   "atom_kv4_extend")
    return slots, q_start, lens_out, state_out


def atom_kv4_release(done, lens, table, pool, page, lens_out=None, state_out=None, stream=None):
    """Give the pages of the sequences with done[b] (bool [batch]) back to the pool, whose `free` is written behind its free
    pages.  Returns (lens_out, state_out): lengths, 0 where done, and the pool's new state; either may be given as its input,
    which is then replaced (more than 64 sequences take a second launch for it)."""
    free, state = _pool(pool)
    page = _bq._size(page, "page")
    if stream is None and lens_out is None and state_out is None and _bq._SHORT is not None:
        out = _bq._SHORT.kv4_release(done, lens, table, free, state, page)
        if out is not None:
            return out
    torch = _bq._torch()
    i32 = torch.int32
    batch, width = _bq._mat(table, "table")
    lens_out = empty((batch,), i32, table, stream) if lens_out is None else lens_out
    state_out = empty((2,), i32, table, stream) if state_out is None else state_out
    p = _bq._ptrs((done, "done", torch.bool, (batch,)), (lens, "lens", i32, (batch,)), (table, "table", i32, (batch, width)),
                  (free, "free", i32, None), (state, "state", i32, (2,)), (lens_out, "lens_out", i32, (batch,)),
                  (state_out, "state_out", i32, (2,)))
    with on_device(table):
        _bq._check(_bq.load_library().atom_kv4_release(p[0], p[1], p[2], batch, width, page, p[3], _bq._c_int(free.shape[0]), p[4],
                                                       p[5], p[6], _bq._stream(stream, table.device)), "atom_kv4_release")
    return lens_out, state_out
