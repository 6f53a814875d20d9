"""The norm's exact steps, evaluated on the host (norm_steps.h is plain arithmetic)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_quantized_gemm_amd", "csrc")


def run(tmp_path, text):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    (tmp_path / "t.cpp").write_text(text)
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-ffp-contract=off", "-I" + CSRC, str(tmp_path / "t.cpp"), "-o",
                    str(tmp_path / "t")], check=True)
    return subprocess.run([str(tmp_path / "t")], capture_output=True, text=True, check=True).stdout.split()


DIVIDED = r"""
#include <math.h>
#include <stdio.h>
#include <random>
#include "norm_steps.h"
static long bad = 0, count = 0, product = 0;
static void check(double a, double b) {
  const double r = 1.0 / b;
  bad += rms::divided(a, b, r) != a / b;
  product += a * r != a / b;
  ++count;
}
int main() {
  std::mt19937_64 g(1);
  auto uniform = [&] { return 1.0 + (double)(g() >> 12) * 0x1p-52; };
  for (int i = 0; i < 3000000; ++i) {
    const float p = (float)((int)(g() % 4194303) + 1) * 0x1p-12f;     // h * w: at most 22 bits
    const double mean = uniform() * ldexp(1.0, (int)(g() % 40) - 20);
    check(p, sqrt(mean));                                             // y
    check(p, sqrt((double)((g() % 99999) + 1)));
    check(uniform(), uniform());
    check(mean, (double)((g() % 65536) + 1));                         // the mean
    check(uniform() * 100, (double)(float)uniform());                 // y / s
    check(uniform(), 127.0);
    check(nextafter(2.0, 1.0), uniform());
    check(uniform(), nextafter(2.0, 1.0));
  }
  for (int c = 1; c < 4096; ++c)                                      // the quotient is a border itself
    for (double w : {0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 62.5, 126.5, 127.0}) check(c * w, c);
  for (int k = 1; k <= 65536; ++k)
    for (double c : {1.0, 49.0, 2401.0, 0.140625}) check(k * c, k);
  // the ends of the rows' range: bf16's smallest and largest products and norms
  for (int i = 0; i < 200000; ++i)
    for (int e : {-149, -100, 100, 127})
      for (int f : {-40, 120}) check(ldexp(uniform(), e), ldexp(uniform(), f));
  printf("%ld %ld %ld\n", bad, count, product);
}
"""


def test_divided_is_the_division(tmp_path):
    """Bit for bit that of the hardware, over the norm's values; a product with the reciprocal is not."""
    bad, count, product = map(int, run(tmp_path, DIVIDED))
    assert count > 2e7 and product > count // 10
    assert bad == 0


BORDERS = r"""
#include <stdio.h>
#include "norm_steps.h"
int main() {                                                          // numbers in, distances out
  float f;
  int step;
  while (scanf("%f %d", &f, &step) == 2) {
    uint32_t b;
    __builtin_memcpy(&b, &f, 4);
    printf("%u\n", rms::border_distance(b + step));
  }
}
"""


def test_borders_are_seen_and_nothing_else(tmp_path):
    """Each border and its neighbours of either sign; no zero, none of the padding's, nothing far from a border."""
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    (tmp_path / "b.cpp").write_text(BORDERS)
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-I" + CSRC, str(tmp_path / "b.cpp"), "-o", str(tmp_path / "b")], check=True)

    def distances(pairs):
        text = "\n".join(f"{f!r} {s}" for f, s in pairs)
        return list(map(int, subprocess.run([str(tmp_path / "b")], input=text, capture_output=True, text=True, check=True).stdout.split()))
    borders = [s * b for b in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0, 8.0) for s in (1.0, -1.0)]
    assert all(d < 8 for d in distances([(b, s) for b in borders for s in range(-4, 4)]))
    assert all(d >= 8 for d in distances([(b, s) for b in borders for s in (-20, -5, 4, 20, 1000)]))
    assert all(d >= 8 for d in distances([(0.0, 0), (-0.0, 0), (1e-30, 0), (0.0625, 0), (0.125, -1), (1.1, 0), (2.9, 0), (5.9, 0)]))
