"""CPU oracle of the MXFP4 layer, the norm in front of the quantized layers and the KV cache's bookkeeping (numpy, fp64 and
exact integers).

Written from the definitions in ``include/atom_mxfp4.h``, ``include/atom_norm.h`` and ``include/atom_kv4_pages.h``; shares no
code with the HIP path.  Inputs are fp32 arrays that hold fp16 or bf16 values exactly.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def mx_row_bytes(K):
    return -(-K // 256) * 128


def mx_codes(x):
    """(codes uint8 [rows, padded K], scale bytes uint8 [rows, padded K / 32]) of fp32 or fp64 rows, unpacked."""
    x = np.asarray(x, np.float64)
    rows, K = x.shape
    p = np.zeros((rows, 2 * mx_row_bytes(K)))
    p[:, :K] = x
    b = p.reshape(rows, -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    e = np.where(top > 0, np.frexp(top)[1] - 1 - 2, -127).clip(-127, 125)
    u = np.ldexp(b, -e[..., None])
    a = np.abs(u)
    # between neighbours of the grid: the nearer one, the even code where both are as near
    mid = (GRID[1:] + GRID[:-1]) / 2
    code = np.zeros(u.shape, np.int64)
    for i, m in enumerate(mid):                       # the border below code i + 1: it belongs to the even one of i, i + 1
        code += (a >= m) if i % 2 else (a > m)
    code |= np.signbit(u).astype(np.int64) << 3
    code[bad] = 0
    return code.reshape(rows, -1).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def mx_pack(codes, scales):
    """The packed arrays (uint8 [rows, row bytes], uint8 [groups, rows, 8])."""
    rows = codes.shape[0]
    return codes[:, 0::2] | (codes[:, 1::2] << 4), np.ascontiguousarray(scales.reshape(rows, -1, 8).transpose(1, 0, 2))


def mx_unpack(q, s):
    rows = q.shape[0]
    codes = np.stack([q & 15, q >> 4], -1).reshape(rows, -1)
    return codes, s.transpose(1, 0, 2).reshape(rows, -1)


def mx_values(codes, scales):
    """fp64 values [rows, padded K] of unpacked codes."""
    v = np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7]
    e = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(e, 32, -1)


def rmsnorm(x, w, eps, residual=None, to16=None):
    """(y fp64, h fp32) of fp32 rows; `to16` rounds fp32 values to the rows' type."""
    x = np.asarray(x, np.float32)
    h = x if residual is None else to16(x + np.asarray(residual, np.float32))
    d = h.astype(np.float64)
    return d * np.asarray(w, np.float64) / np.sqrt((d * d).mean(1, keepdims=True) + eps), h


def w8_codes(y):
    """(codes int8 [rows, row bytes], scales fp32) of fp64 rows."""
    rows, K = y.shape
    s = (np.abs(y).max(1) / 127).astype(np.float32)
    q = np.zeros((rows, -(-K // 128) * 128), np.int8)
    live = s > 0
    q[live, :K] = np.clip(np.rint(y[live] / s[live, None].astype(np.float64)), -127, 127).astype(np.int8)
    return q, s


def extend(lens, new, table, free, state, page, total):
    """A step's tokens, one by one: (slots, start, lens, table, state)."""
    batch, width = table.shape
    most = width * page
    lens, table, pool = [min(max(int(n), 0), most) for n in lens], table.copy(), min(max(int(state[0]), 0), len(free))
    start, rows = [0], 0
    for n in new:
        rows = min(rows + max(int(n), 0), total)
        start.append(rows)
    slots, at, pages, out = np.full(total, -1, np.int64), pool, table.copy(), []
    needed = 0
    for b in range(batch):
        t = lens[b]
        held = -(-t // page)
        for r in range(start[b], start[b + 1]):
            if t < most:
                if t // page >= held:
                    needed += 1
                    at -= 1
                    if at >= 0:
                        pages[b, held] = free[at]
                    held += 1
                if at >= 0 and pages[b, t // page] >= 0:
                    slots[r] = int(pages[b, t // page]) * page + t % page
                t += 1
        out.append(t)
    if needed > pool:
        return np.full(total, -1, np.int64), np.array(start), np.array(lens), table, np.array([pool, needed - pool])
    return slots, np.array(start), np.array(out), pages, np.array([pool - needed, 0])


def release(done, lens, table, free, state, page):
    """(lens, free, state) behind the sequences that are done."""
    batch, width = table.shape
    free, pool = free.copy(), min(max(int(state[0]), 0), len(free))
    lens = [min(max(int(n), 0), width * page) for n in lens]
    for b in range(batch):
        if done[b]:
            for c in range(-(-lens[b] // page)):
                if pool < len(free):
                    free[pool] = table[b, c]
                    pool += 1
            lens[b] = 0
    return np.array(lens), free, np.array([pool, 0])
