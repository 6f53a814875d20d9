"""Pins of the CPU oracle of the W8A8 layer and the KV cache: hand-derived codes and bytes, closed-form
bounds, and the C layout helpers walked over good and bad inputs (no GPU)."""
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import serve_oracle as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_w8a8_codes_by_hand():
    # max 254: scale 2; 3 / 2 = 1.5 -> 2 (even), 5 / 2 = 2.5 -> 2 (even), -7 / 2 = -3.5 -> -4 (even), 1 / 2 = 0.5 -> 0
    q, s = S.quantize_w8a8(np.array([[254, 3, 5, -7, 1, -254], [0, 0, 0, 0, 0, 0]], np.float32))
    assert s.tolist() == [2.0, 0.0]
    assert q.shape == (2, 128)
    assert q[0, :6].tolist() == [127, 2, 2, -4, 0, -127] and not q[0, 6:].any() and not q[1].any()


def test_w8a8_round_trip_and_product():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((7, 200)).astype(np.float16).astype(np.float32)
    w = rng.standard_normal((5, 200)).astype(np.float16).astype(np.float32)
    (qx, sx), (qw, sw) = S.quantize_w8a8(x), S.quantize_w8a8(w)
    assert np.all(np.abs(x - qx[:, :200] * sx[:, None]) <= sx[:, None] * (0.5 + 2.0**-16))
    assert np.all(np.abs(qx).max(1) == 127)
    y, _ = S.gemm_w8a8(qx, sx, qw, sw)
    want = [[sum(int(a) * int(b) for a, b in zip(qx[m], qw[n])) * float(sx[m]) * float(sw[n]) for n in range(5)]
            for m in range(7)]
    np.testing.assert_allclose(y, want, rtol=1e-14)


def test_kv4_codes_by_hand():
    # [-3, 12]: scale 1, zero 3: 0.5 -> 0 + 3, 1.5 -> 2 + 3, -0.5 -> 0 + 3, -2.5 -> -2 + 3
    q, z, s = S.kv4_quantize(np.array([[-3, 12, 0.5, 1.5, -0.5, -2.5, 0, 11.4]], np.float32))
    assert (z[0], s[0]) == (3, 1) and q[0].tolist() == [0, 15, 3, 5, 3, 1, 3, 14]
    # all positive: the range starts at 0; a constant row keeps its value
    q, z, s = S.kv4_quantize(np.full((1, 4), 30, np.float32))
    assert (z[0], s[0]) == (0, 2) and q[0].tolist() == [15] * 4
    q, z, s = S.kv4_quantize(np.zeros((1, 4), np.float32))
    assert (z[0], s[0]) == (0, 0) and not q.any()
    # a scale below half of fp16's smallest number is 0
    q, z, s = S.kv4_quantize(np.full((1, 4), 2.0**-23, np.float32))
    assert s[0] == 0 and not q.any()
    # beyond fp16: the scale saturates
    q, z, s = S.kv4_quantize(np.array([[1e30, -1e30]], np.float32))
    assert s[0] == 65504 and z[0] == 15 and q[0].tolist() == [15, 0]


def test_kv4_round_trip_bound():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((64, 3, 64)).astype(np.float16).astype(np.float32)
    q, z, s = S.kv4_quantize(x)
    err = np.abs((q - z[..., None]) * s[..., None] - x)
    # half a step inside the range; at its ends the zero point's own rounding costs up to half a step more, and the
    # scale's rounding (2^-11) up to 15 of that
    assert np.all(err <= s[..., None] * (1.0 + 15 * 2.0**-11 + 1e-6))
    assert np.mean(err <= s[..., None] * 0.5001) > 0.95


def _arrays(pages, H, page, D, fill):
    return (np.full((pages, H, page, D // 2), fill, np.uint8), np.zeros((pages, H, page, 2), np.float16),
            np.full((pages, H, page // 4, D // 4, 8), fill, np.uint8), np.zeros((pages, H, page, 2), np.float16))


def test_kv4_bytes_by_hand():
    cache = _arrays(2, 1, 16, 64, 0)
    codes = (np.arange(64) % 16).astype(np.uint8).reshape(1, 1, 64)
    one = np.ones((1, 1), np.float32)
    S.kv4_write(cache, 16, [16 + 6], 0, codes, 3 * one, 0.5 * one)
    S.kv4_write(cache, 16, [16 + 6], 1, codes, 3 * one, 0.5 * one)
    assert cache[0][1, 0, 6, :4].tolist() == [0x10, 0x32, 0x54, 0x76]
    # token 6 = block 1, third token: bytes 4 and 5 of each channel quad
    assert cache[2][1, 0, 1, 0].tolist() == [0, 0, 0, 0, 0x10, 0x32, 0, 0]
    assert cache[2][1, 0, 1, 1].tolist() == [0, 0, 0, 0, 0x54, 0x76, 0, 0]
    assert cache[1][1, 0, 6].tolist() == [3.0, 0.5]
    for side in (0, 1):
        np.testing.assert_array_equal(S.kv4_read(cache, 16, [22, -1, 32], side)[0, 0], (codes[0, 0] - 3.0) * 0.5)
        assert not S.kv4_read(cache, 16, [-1, 32], side).any()


def test_kv4_every_slot_has_its_own_nibbles():
    cache = _arrays(1, 2, 16, 64, 0xAB)
    rng = np.random.default_rng(3)
    codes = rng.integers(0, 16, (2, 16, 2, 64)).astype(np.uint8)
    one = np.ones((16, 2), np.float32)
    order = rng.permutation(16)
    for side in (0, 1):
        S.kv4_write(cache, 16, order, side, codes[side][order], 0 * one, one)
    for side in (0, 1):
        np.testing.assert_array_equal(S.kv4_read(cache, 16, np.arange(16), side), codes[side])


def test_attention_against_a_loop():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((2, 2, 8)), rng.standard_normal((2, 2, 8))
    out, _, _ = S.attention(q, k, v, 0.3)
    assert not out[0].any()                        # two tokens, three queries: the first sees none
    np.testing.assert_allclose(out[1], np.repeat(v[0], 2, 0))
    for j in range(4):
        e = [np.exp(0.3 * float(np.dot(q[2, j], k[t, j // 2]))) for t in range(2)]
        np.testing.assert_allclose(out[2, j], (e[0] * v[0, j // 2] + e[1] * v[1, j // 2]) / sum(e), rtol=1e-12)


LAYOUT = r"""
#include <limits.h>
#include <stdio.h>
#include "kv4_layout.h"
#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
int main() {
  const int bad[] = {INT_MIN, -1, 0, 1, 5, 6, 7, 1000000000, INT_MAX};
  const int n = sizeof(bad) / sizeof(bad[0]);
  for (int i = 0; i < n; ++i) {
    const int p = kv4::page_id(bad[i], 6);
    CHECK(p >= 0 && p < 6 && (bad[i] < 0 || bad[i] >= 6 || p == bad[i]));
    for (int len = 0; len < n; ++len)
      for (int e = 0; e < n; ++e) {
        const kv4::Sequence s = kv4::sequence(bad[i], bad[e], bad[len], 6, 4, 100, 64);
        CHECK(s.first >= 0 && s.queries >= 0 && s.first + s.queries <= 6 && s.queries <= 4 && s.behind >= s.queries);
        CHECK(s.tokens >= 0 && s.tokens <= 64);
        for (int q = 0; q < s.queries; ++q) CHECK(kv4::visible(s, q) >= 0 && kv4::visible(s, q) <= s.tokens);
      }
  }
  const kv4::Sequence s = kv4::sequence(2, 5, 10, 6, 4, 100, 64);
  CHECK(s.first == 2 && s.queries == 3 && s.tokens == 10 && kv4::visible(s, 0) == 8 && kv4::visible(s, 2) == 10);
  CHECK(kv4::visible(kv4::sequence(0, 3, 1, 6, 4, 100, 64), 0) == 0);
  CHECK(kv4::visible(kv4::sequence(0, 6, 9, 6, 4, 100, 64), 0) == 4);     // six queries, four of them run
  for (int t = 0; t < 64 + 40; ++t) {
    const int c = kv4::table_column(t, 4, 4);
    CHECK(c >= 0 && c < 4 && (t >= 64 || c == t / 16));
  }
  const int64_t slots[] = {INT64_MIN, -1, 0, 95, 96, (int64_t)1 << 40, INT64_MAX};
  const bool in[] = {false, false, true, true, false, false, false};
  for (int i = 0; i < 7; ++i) CHECK(kv4::valid_slot(slots[i], 6, 4) == in[i]);
  // past 32 bits: the last token of a pool of 2^22 pages of 256 tokens and 8 heads
  CHECK(kv4::row_index((1 << 22) - 1, 7, 8, 8, 255) == ((int64_t)1 << 33) - 1);
  CHECK(kv4::value_block((1 << 22) - 1, 7, 8, 8, 128, 63) == (((int64_t)1 << 33) - 4) * 64);
  // a block's tokens and quads tile its bytes
  unsigned char seen[256] = {0};
  for (int quad = 0; quad < 32; ++quad)
    for (int t = 0; t < 4; ++t)
      for (int b = 0; b < 2; ++b) CHECK(!seen[kv4::value_in_block(quad, t) + b]++);
  printf("ok\n");
  return 0;
}
"""


def test_layout_clamps(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    src = tmp_path / "layout.cpp"
    src.write_text(LAYOUT)
    exe = tmp_path / "layout"
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-Wno-unused-function",
                    f"-I{os.path.join(ROOT, 'bit_quantized_gemm_amd', 'csrc')}", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout
