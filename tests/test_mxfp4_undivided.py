"""MXFP4 products that are given no scratch memory: the plan is one for that, not a divided one's kernel run whole (no GPU needed;
mxfp4_plan.h is plain arithmetic)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MAIN = r"""
#include <stdio.h>
#include "mxfp4_plan.h"
int main() {
  int a[3];                                    // M N K
  while (scanf("%d %d %d", a, a + 1, a + 2) == 3) {
    const atom::mx::Plan p = atom::mx::plan(a[0], a[1], a[2], 256);
    const long long need = atom::mx::part_bytes(p);
    const long long given[3] = {0, need - 1, need};
    printf("%d %d %d %lld", p.kind, p.tiles, p.splits, need);
    for (long long g : given) {
      const atom::mx::Plan q = atom::mx::plan_within(a[0], a[1], a[2], 256, g);
      printf(" %d %d %d %lld", q.kind, q.tiles, q.splits, (long long)atom::mx::part_bytes(q));
    }
    printf("\n");
  }
  return 0;
}
"""

# Us of products of long K, run whole by each kind of kernel (graph replays, operands from HBM; kinds 0 and 1: 16 and 32
# tokens, from 2 up the tiles).
WHOLE = {(64, 4096, 11008): (25.4, 21.3, 25.1, 27.8, 33.6, 38.9, 56.9), (64, 4096, 8192): (19.7, 15.8, 19.9, 22.0, 26.3, 30.7, 45.1),
         (100, 260, 65536): (34.6, 50.2, 125.6, 135.7, 189.6, 198.6, 293.4), (333, 512, 28672): (46.3, 47.2, 61.3, 62.6, 85.8, 101.0, 161.8),
         (200, 1024, 14336): (31.7, 25.6, 31.6, 32.7, 43.8, 52.2, 81.3), (512, 1024, 8192): (34.2, 26.6, 17.8, 19.9, 24.3, 31.8, 51.1)}


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
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


def test_scratch_decides(plans):
    """With enough scratch the plan of the shape, with a byte less or none an undivided one."""
    shapes = [(m, n, k) for m in (1, 17, 64, 100, 333, 777, 2048) for n in (64, 260, 1024, 4096, 11008) for k in (256, 2048, 8192, 14336, 65536)]
    divided = 0
    for s, p in zip(shapes, plans(shapes)):
        best, none, less, enough = p[:4], p[4:8], p[8:12], p[12:]
        assert enough == best, s
        assert none[2] == 1 and none[3] == 0 and none[1] > 0, s
        if best[2] == 1:
            assert none == best, s
        else:
            assert less == none, s
            divided += 1
    assert divided > 20


def test_the_choice_without_scratch(plans):
    """Within a fifth of the fastest kernel measured."""
    for (s, us), p in zip(WHOLE.items(), plans(list(WHOLE))):
        assert us[p[4]] <= 1.2 * min(us), (s, p)


# Us of 64 x 64 tiles whole, and K divided two, three and four ways (as above), where a unit holds one workgroup of the whole product.
DIVIDED = {(777, 777, 8192): (20.2, 17.3, 15.5, 17.0), (777, 777, 7000): (17.1, 15.7, 14.3, 15.7), (64, 4096, 8192): (19.9, 15.3, 13.6, 13.2),
           (64, 4096, 11008): (25.1, 18.3, 15.6, 14.5), (160, 4096, 8192): (19.8, 18.3, 20.6, 20.0), (512, 1024, 8192): (17.8, 15.1, 14.5, 14.2),
           (1024, 512, 11008): (25.4, 18.6, 18.4, 16.7), (333, 512, 28672): (61.3, 36.0, 26.8, 22.5), (200, 1024, 14336): (31.6, 20.7, 16.8, 15.0)}


def test_long_products_are_divided(plans):
    """A lone workgroup a unit waits for HBM at every stage: the division that is chosen is within 15% of the best measured."""
    for (s, us), p in zip(DIVIDED.items(), plans(list(DIVIDED))):
        assert p[0] == 2 and us[p[2] - 1] <= 1.15 * min(us), (s, p)
