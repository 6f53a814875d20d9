"""Pins of the oracle of the MXFP4 layer, the norm and the KV cache's bookkeeping: values derived by hand, a search over the
whole grid, exact rationals, a plain serving loop."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import layer_oracle as O


def test_worked_block():
    """Largest 7.0: e = 2 - 2 = 0, scale byte 127.  Ties go to the even code, 7 saturates to 6, signs of zeros stay."""
    x = np.zeros((1, 32), np.float32)
    x[0, :16] = [7, 0.25, -0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -5, 5.01, 0.26, -0.74, 1.24, 6, -0.0, 0.5]
    c, s = O.mx_codes(x)
    assert s[0].tolist() == [127] + [0] * 7
    assert c[0, :16].tolist() == [7, 0, 8, 2, 2, 4, 4, 6, 14, 7, 1, 9, 2, 7, 8, 1] and not c[0, 16:].any()
    q, s3 = O.mx_pack(c, s)
    assert q.shape == (1, 128) and s3.shape == (1, 1, 8)
    assert q[0, :8].tolist() == [0x07, 0x28, 0x42, 0x64, 0x7E, 0x91, 0x72, 0x18]


@pytest.mark.parametrize("top,byte", [(1.0, 125), (0.999, 124), (3.9, 126), (4.0, 127), (2.0**-24, 101), (65504.0, 140), (2.0**-133, 0),
                                      (2.0**-125, 0), (2.0**-124, 1), (3.0e38, 252), (0.0, 0)])
def test_scale_bytes(top, byte):
    x = np.zeros((1, 32), np.float32)
    x[0, 3] = top
    assert O.mx_codes(x)[1][0, 0] == byte


def test_codes_are_the_nearest():
    r = np.random.default_rng(1)
    x = (r.normal(size=(40, 64)) * 2.0 ** r.integers(-10, 10, (40, 1))).astype(np.float32)
    c, s = O.mx_codes(x)
    v = O.mx_values(c, s)
    for i in range(40):
        for k in range(64):
            step = Fraction(2) ** (int(s[i, k // 32]) - 127)
            far = [abs(Fraction(float(x[i, k])) - sign * Fraction(float(g)) * step) for g in O.GRID for sign in (1, -1)]
            assert abs(Fraction(float(x[i, k])) - Fraction(float(v[i, k]))) == min(far)
    assert np.abs(v).max(1).min() > 0
    # the largest of a block lies in [4, 8) of its scale
    u = np.abs(x.reshape(40, 2, 32)).max(-1) / np.ldexp(1.0, s[:, :2].astype(int) - 127)
    assert (u >= 4).all() and (u < 8).all()


def test_pack_round_trip_and_bad_blocks():
    r = np.random.default_rng(2)
    x = r.normal(size=(5, 300)).astype(np.float32)
    x[2, 40] = np.nan
    x[3, 299] = -np.inf
    c, s = O.mx_codes(x)
    a, b = O.mx_unpack(*O.mx_pack(c, s))
    assert np.array_equal(a, c) and np.array_equal(b, s)
    assert (s == 255).sum() == 2 and s[2, 1] == 255 and s[3, 9] == 255
    assert not c[2, 32:64].any() and not c[3, 288:].any()
    assert [O.mx_row_bytes(k) for k in (1, 256, 257, 4096)] == [128, 128, 256, 2048]
    v = O.mx_values(c, s)
    assert np.isnan(v[2, 32:64]).all() and np.isfinite(np.delete(v, [2, 3], 0)).all()


def test_norm_by_rationals():
    x = np.array([[3, -4, 0, 0], [1, 1, 1, 1]], np.float32)
    w = np.array([1, 2, 3, -0.5], np.float32)
    y, h = O.rmsnorm(x, w, 0.0)
    np.testing.assert_allclose(y, [[3 / 2.5, -8 / 2.5, 0, 0], [1, 2, 3, -0.5]], rtol=1e-15)
    assert np.array_equal(h, x)
    q, s = O.w8_codes(y)
    assert s.tolist() == [np.float32(3.2 / 127), np.float32(3 / 127)] and q.shape == (2, 128)
    assert q[0, :4].tolist() == [48, -127, 0, 0] and q[1, :4].tolist() == [42, 85, 127, -21]
    # the sum is rounded to the rows' type before anything else
    y, h = O.rmsnorm(np.array([[2048.0, 1]], np.float32), w[:2], 1e-6, np.array([[1.0, 0]], np.float32),
                     lambda v: v.astype(np.float16).astype(np.float32))
    assert h.tolist() == [[2048.0, 1.0]]


def test_extend_by_hand():
    """Two sequences of pages of 16: 15 + 3 tokens take the rest of page 5 and the pool's last; 0 + 17 two more."""
    table = np.array([[5, -1, -1], [9, 9, 9]])
    free = np.array([7, 8, 2, 3])
    got = O.extend([15, 0], [3, 17], table, free, [4, 0], 16, 22)
    slots = [5 * 16 + 15, 3 * 16, 3 * 16 + 1] + [2 * 16 + i for i in range(16)] + [8 * 16] + [-1, -1]
    assert got[0].tolist() == slots and got[1].tolist() == [0, 3, 20] and got[2].tolist() == [18, 17]
    assert got[3].tolist() == [[5, 3, -1], [2, 8, 9]] and got[4].tolist() == [1, 0]
    short = O.extend([15, 0], [3, 17], table, free, [2, 0], 16, 22)
    assert (short[0] == -1).all() and short[2].tolist() == [15, 0] and np.array_equal(short[3], table) and short[4].tolist() == [2, 1]
    lens, back, st = O.release([True, False], got[2], got[3], free, got[4], 16)
    assert lens.tolist() == [0, 17] and back.tolist() == [7, 5, 3, 3] and st.tolist() == [3, 0]


def test_serving_loop_keeps_its_pages():
    r = np.random.default_rng(3)
    pages, batch, width = 40, 6, 8
    free, st = np.arange(pages), np.array([pages, 0])
    lens, table = np.zeros(batch, int), np.full((batch, width), -1)
    for step in range(50):
        new = np.minimum(r.integers(0, 20, batch), width * 16 - lens)
        _, _, lens, table, st = O.extend(lens, new, table, free, st, 16, 200)
        lens, free, st = O.release(r.random(batch) < 0.2, lens, table, free, st, 16)
        held = table[np.arange(width) < -(-lens // 16)[:, None]]
        assert sorted(held.tolist() + free[:st[0]].tolist()) == list(range(pages))
