"""The divide-free quotient of the W8A8 and KV cache quantizers, walked over every pair of significands on the CPU.

q = x r, u = fma(fma(-q, s, x), r, q) with r = fl32(1 / s): the nearest integer of u must be that of fl32(x / s), ties to
even.  Everything but the exponents' ends is scale-free, so one binade of scales and the binades of x whose quotients
reach 1/4 to 32 (KV cache) or 1/4 to 127 (W8A8) stand for all.  80-bit floats hold each fma's exact sum (48 bits and a 24-bit
addend that overlaps them)."""
import numpy as np
import pytest

L = np.longdouble


def once_corrected(x, s, r):
    q = (x * r).astype(np.float32)
    e = (L(0) + x - q.astype(L) * s.astype(L)).astype(np.float32)
    return (e.astype(L) * r.astype(L) + q).astype(np.float32)


@pytest.mark.parametrize("bits", [8, 11])
def test_w8a8_quotients(bits):
    one = 1 << (bits - 1)
    sig = np.arange(one, 2 * one)
    for a in sig:                                                # the row's maximum
        s = np.float32(a) / np.float32(127)
        x = np.concatenate([sig * 2.0**-e for e in range(9)])
        x = x[x <= a].astype(np.float32)
        s = np.full_like(x, s)
        u = once_corrected(x, s, np.float32(1) / s)
        np.testing.assert_array_equal(np.rint(u), np.rint(x / s))
        assert np.rint(u).max() == 127


@pytest.mark.parametrize("bits", [8, 11])
def test_kv4_quotients(bits):
    one = 1 << (bits - 1)
    x = np.concatenate([np.arange(one, 2 * one) / one * 2.0**e for e in range(-3, 6)]).astype(np.float32)
    for k in range(1024):                                        # every fp16 significand
        s = np.full_like(x, 1 + k / 1024)
        u = once_corrected(x, s, np.float32(1) / s)
        np.testing.assert_array_equal(np.rint(u), np.rint(x / s))


def test_fifteenths():
    """fl32(d / 15) by two corrected steps, then fp16: over random ranges and those next to fp16's rounding borders."""
    rng = np.random.default_rng(0)
    h = np.arange(1, 0x7C00, dtype=np.uint16).view(np.float16).astype(np.float64)
    border = np.concatenate([(h[1:] + h[:-1]) / 2 * 15, h * 15])
    d = np.concatenate([border * (1 + k * 2.0**-24) for k in range(-3, 4)] + [np.exp(rng.uniform(-20, 12, 1000000))])
    d = d.astype(np.float32)
    r = np.full_like(d, np.float32(1) / np.float32(15))
    s = np.full_like(d, 15)
    d0 = (d * r).astype(np.float32)
    for _ in range(2):
        e = (L(0) + d - d0.astype(L) * s.astype(L)).astype(np.float32)
        d0 = (e.astype(L) * r.astype(L) + d0).astype(np.float32)
    np.testing.assert_array_equal(d0, d / s)
