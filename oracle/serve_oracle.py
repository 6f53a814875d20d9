"""CPU oracle of the W8A8 layer and the 4-bit KV cache (numpy, exact integers and fp64).

Written from the definitions in ``include/atom_w8a8.h`` and ``include/atom_kv4.h``; shares no code with
the HIP path.  Inputs are fp32 arrays that hold fp16 or bf16 values exactly.
"""
from __future__ import annotations

import numpy as np


def row_bytes(K):
    return -(-K // 128) * 128


def quantize_w8a8(x):
    """(codes int8 [rows, row bytes], scales fp32 [rows]) of fp32 rows."""
    x = np.asarray(x, np.float32)
    rows, K = x.shape
    s = (np.abs(x).max(1) / np.float32(127)).astype(np.float32)
    q = np.zeros((rows, row_bytes(K)), np.int8)
    live = s > 0
    q[live, :K] = np.clip(np.rint(x[live] / s[live, None]), -127, 127).astype(np.int8)
    return q, s


def gemm_w8a8(qx, sx, qw, sw, bias=None):
    """fp64 Y of packed operands, and |acc * sx * sw| (for error bounds)."""
    acc = qx.astype(np.float64) @ qw.astype(np.float64).T        # integers below 2^53: exact
    y = acc * sx.astype(np.float64)[:, None] * sw.astype(np.float64)[None]
    mag = np.abs(y)
    return (y if bias is None else y + bias.astype(np.float64)[None]), mag


def kv4_quantize(x):
    """(codes, zero, scale) of fp32 rows x [..., D]; zero and scale [...] as fp32 values of fp16."""
    x = np.asarray(x, np.float32)
    lo, hi = np.minimum(x.min(-1), 0), np.maximum(x.max(-1), 0)
    with np.errstate(over="ignore"):
        s = np.minimum((hi - lo) / np.float32(15), np.float32(65504)).astype(np.float16).astype(np.float32)
    live = s > 0
    d = np.where(live, s, 1).astype(np.float32)
    zero = np.where(live, np.clip(np.rint(-lo / d), 0, 15), 0).astype(np.float32) + np.float32(0)   # never -0
    q = np.clip(np.rint(x / d[..., None]) + zero[..., None], 0, 15)
    return np.where(live[..., None], q, 0).astype(np.uint8), zero, s


def kv4_write(cache, page, slots, side, codes, zero, scale):
    """Codes [tokens, H, D] and parameters into numpy cache arrays (k, k_par, v, v_par), byte by byte as the
    header places them.  side: 0 keys, 1 values."""
    arr, par = (cache[0], cache[1]) if side == 0 else (cache[2], cache[3])
    D = codes.shape[-1]
    d = np.arange(D)
    for i, slot in enumerate(slots):
        if slot < 0 or slot // page >= arr.shape[0]:
            continue
        p, t = slot // page, slot % page
        par[p, :, t, 0], par[p, :, t, 1] = zero[i], scale[i]
        for nib in (0, 1):
            c = codes[i][:, d % 2 == nib]
            e = d[d % 2 == nib]
            mask, shift = (0xF0, 0) if nib == 0 else (0x0F, 4)
            if side == 0:
                arr[p, :, t, e // 2] = ((arr[p, :, t, e // 2].T & mask) | (c << shift)).T
            else:
                at = (p, slice(None), t // 4, e // 4, 4 * ((t % 4) // 2) + 2 * (t % 2) + (e % 4) // 2)
                arr[at] = ((arr[at].T & mask) | (c << shift)).T


def kv4_read(cache, page, slots, side):
    """fp64 values [tokens, H, D] of the codes in `slots`."""
    arr, par = (cache[0], cache[1]) if side == 0 else (cache[2], cache[3])
    H = arr.shape[1]
    D = arr.shape[3] * (2 if side == 0 else 4)
    d = np.arange(D)
    out = np.zeros((len(slots), H, D))
    for i, slot in enumerate(slots):
        if slot < 0 or slot // page >= arr.shape[0]:
            continue
        p, t = slot // page, slot % page
        if side == 0:
            b = arr[p, :, t][:, d // 2]
        else:
            b = arr[p, :, t // 4][:, d // 4, 4 * ((t % 4) // 2) + 2 * (t % 2) + (d % 4) // 2]
        c = np.where(d % 2 == 0, b & 15, b >> 4).astype(np.float64)
        z, s = par[p, :, t, 0].astype(np.float64), par[p, :, t, 1].astype(np.float64)
        out[i] = (c - z[:, None]) * s[:, None]
    return out


def attention(q, key, value, scale):
    """Causal attention of the last queries of one sequence in fp64: q [n, Hq, D], key / value [tokens, H, D].
    Returns (out, weights' mean of |value|, largest sum of |scale q k| of a query and a token in sight)."""
    n, Hq, D = q.shape
    tokens, H, _ = key.shape
    out, mag, big = np.zeros((n, Hq, D)), np.zeros((n, Hq, D)), np.zeros((n, Hq))
    for i in range(n):
        seen = tokens - n + i + 1
        if seen <= 0:
            continue
        for j in range(Hq):
            k, v = key[:seen, j // (Hq // H)], value[:seen, j // (Hq // H)]
            s = scale * (k @ q[i, j])
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, j], mag[i, j] = w @ v, w @ np.abs(v)
            big[i, j] = scale * (np.abs(k) @ np.abs(q[i, j])).max()
    return out, mag, big
