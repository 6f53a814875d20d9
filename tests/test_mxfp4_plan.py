"""The launch plan of MXFP4 products, evaluated on the host (mxfp4_plan.h is plain arithmetic)."""
import os
import shutil
import subprocess

import pytest

import bit_quantized_gemm_amd as bq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TILES = {2: (64, 64), 3: (64, 128), 4: (128, 128), 5: (256, 128), 6: (256, 256)}
MAIN = r"""
#include <stdio.h>
#include "mxfp4_plan.h"
int main() {
  int a[3];                                    // M N K
  while (scanf("%d %d %d", a, a + 1, a + 2) == 3) {
    const atom::mx::Plan p = atom::mx::plan(a[0], a[1], a[2], 256);
    const bool one = atom::mx::rows_fit(a[0], a[1], a[2], 256);
    const atom::mx::RowsPlan r = one ? atom::mx::rows_plan(a[0], a[1], a[2], 256) : atom::mx::RowsPlan{0, 0};
    printf("%d %d %d %d %d %d\n", p.kind, p.tiles, p.splits, atom::mx::rows_waves((a[2] + 255) / 256), r.columns, r.waves);
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """A function from shapes (M, N, K) to their (kind, tiles, splits, waves of a few-rows workgroup, and of one launch: times
    16 columns, or 0 where it takes two, and waves)."""
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(MAIN)
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-I" + os.path.join(ROOT, "bit_quantized_gemm_amd", "csrc"),
                    str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)

    def run(shapes):
        text = "\n".join(" ".join(map(str, s)) for s in shapes)
        out = subprocess.run([str(d / "plan")], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return run


def test_plans_fit_a_launch(plans):
    """Every shape whose output fits 2^40 bytes gets a plan with all its tiles and less than 2^32 threads; K is divided
    only where each part has four groups."""
    sizes = [1, 2, 15, 16, 17, 33, 64, 65, 128, 129, 300, 1000, 4096, 11008, 65535, 65536, 1 << 17, (1 << 20) - 1, 1 << 20, (1 << 20) + 1,
             1 << 22, (1 << 24) - 1, 1 << 24]
    shapes = [(m, n, k) for m in sizes for n in sizes for k in (1, 256, 257, 1024, 4096, 11008, 65536)
              if m * n <= 1 << 39 and -(-m // 128) * -(-n // 128) <= 1 << 26]
    for (M, N, K), (kind, tiles, splits, waves, _, _) in zip(shapes, plans(shapes)):
        bm, bn = TILES.get(kind, (16 * (kind + 1), 16))
        assert tiles == -(-M // bm) * -(-N // bn) > 0, (M, N, K)
        assert tiles * splits * (64 * waves if kind < 2 else 256) < 1 << 32
        assert kind >= 2 or -(-M // bm) < 65536
        assert splits == 1 or (kind == 2 and splits <= 4 and -(-K // 256) >= 4 * splits and tiles * splits <= 3 * 256)
        assert 4 <= waves <= 16


def test_one_launch_fits_lds(plans):
    """Sums, codes and scales of the tokens that one launch takes stay within 64 KB for every K, and its tiles in a grid."""
    shapes = [(m, n, k) for m in (*range(1, 18), 33, 256, 333, 1000, 4096, 4097, 1 << 24) for n in (1, 64, 65, 777, 784, 4096, 11008, 16384, 16385, 1 << 20, 1 << 24)
              for k in (1, 256, 257, 4095, 4096, 4097, 8192, 10922, 10923, 16384, 16385, 32768, 65536)]
    for (M, N, K), (_, _, _, _, columns, waves) in zip(shapes, plans(shapes)):
        pairs = (-(-K // 256) + 1) // 2
        tokens, blocks = min(M, 16), -(-M // 16)
        round_ = -(-N // 64) * blocks <= 256 or (K <= 2048 and -(-N // 48) * blocks <= 384)
        assert (columns > 0) == (M == 1 or (tokens * K <= 65536 and (M <= 8 or round_))), (M, N, K)
        if columns:
            assert M <= 8 or -(-N // (16 * columns)) * blocks <= (384 if columns == 3 and K <= 2048 else 256)
            assert columns <= 4 and waves in (4, 8, 12, 16)
            assert max(waves * columns * 1024, tokens * (pairs * 272 + 20)) <= 65536, (M, N, K)
            assert -(-N // (16 * columns)) * 64 * waves < 1 << 32


def test_the_kernel_of_each_tested_shape(plans):
    """The GPU tests' shapes reach every kernel, every division of K, and every ending of each ring of stage buffers."""
    from test_gpu_mxfp4 import ONE, RINGS, SHAPES
    got = plans(SHAPES)
    assert {p[0] for p in got} == set(range(7))
    assert {p[2] for p in got if p[0] == 2} == {1, 2, 3, 4}
    ends = {}
    for (_, _, g), p in zip(RINGS, plans([(m, n, 256 * g - 5) for m, n, g in RINGS])):
        assert p[2] == 1
        ends.setdefault(p[0], set()).add(g)
    assert {g % 6 for g in ends[2]} == {g % 6 for g in ends[3]} == {g % 6 for g in ends[5]} == set(range(6))
    assert {g % 2 for g in ends[4]} == {g % 2 for g in ends[6]} == {0, 1}
    assert min(ends[2]) == min(ends[3]) == min(ends[4]) == 1
    one = plans(ONE)
    assert {(p[4], p[5]) for p in one} >= {(c, w) for c in (1, 2, 3, 4) for w in (4, 8)} and {p[5] for p in one} == {4, 8, 12, 16}


def test_workspace_follows_the_plan(plans):
    if not os.path.exists(bq.lib_path()):
        pytest.skip("libatom.so not built (python -m bit_quantized_gemm_amd.build)")
    shapes = [(64, 4096, 8192), (777, 777, 7000), (16, 4096, 4096), (1024, 11008, 4096), (100, 260, 65536)]
    for (M, N, K), (_, tiles, splits, _, one, _) in zip(shapes, plans(shapes)):
        assert bq.atom_gemm_mxfp4_workspace_bytes(M, N, K) == (splits * tiles * 64 * 64 * 4 if splits > 1 else 0)
        assert bq.atom_linear_mxfp4_workspace_bytes(M, N, K) > bq.atom_gemm_mxfp4_workspace_bytes(M, N, K) or one
