"""The W8A8 row quantize's launches, evaluated on the host (w8a8_rows.h is plain arithmetic)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MAIN = r"""
#include <stdio.h>
#include "w8a8_rows.h"
using namespace atom;
#define CHECK(x) do { if (!(x)) { printf("line %d: %s (rows %lld, K %d)\n", __LINE__, #x, (long long)rows, Kp); return 1; } } while (0)
int main() {
  const int64_t all[] = {1, 384, 385, 1024, 1025, 4000, 1 << 22, 1 << 23, (1 << 24) - 1, 1 << 24};
  for (int64_t rows : all)
    for (int Kp = 128; Kp <= 65536; Kp += 128) {
      const w8a8::RowShape s = w8a8::row_shape(rows, Kp);
      CHECK(s.threads * s.chunks * 8 >= Kp);                        // the row's elements are all held
      const int block = w8a8::block_threads(s.threads), per = block / s.threads;
      CHECK(block <= 1024 && block % s.threads == 0);
      int64_t done = 0;
      int launches = 0;
      while (done < rows) {                                         // as the launcher walks the rows
        const int64_t left = rows - done, n = left < w8a8::launch_rows(s.threads) ? left : w8a8::launch_rows(s.threads);
        CHECK((uint64_t)((n + per - 1) / per) * block < (uint64_t)1 << 32);
        done += n;
        ++launches;
      }
      CHECK(done == rows && launches <= 5 && (rows > 4000 || launches == 1));
    }
  printf("ok\n");
  return 0;
}
"""


def test_no_launch_has_more_threads_than_it_may(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    (tmp_path / "rows.cpp").write_text(MAIN)
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-I" + os.path.join(ROOT, "bit_quantized_gemm_amd", "csrc"),
                    str(tmp_path / "rows.cpp"), "-o", str(tmp_path / "rows")], check=True)
    r = subprocess.run([str(tmp_path / "rows")], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout
