"""The launch plan of attention over the 4-bit KV cache, evaluated on the host (kv4_plan.h is plain arithmetic)."""
import os
import shutil
import subprocess

import pytest

import bit_quantized_gemm_amd as bq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FOUR, EIGHT, PROMPT = 1, 2, 3
MAIN = r"""
#include <stdio.h>
#include "kv4_plan.h"
int main() {
  int a[7];                                    // q_heads heads dim batch max_q max_len cus
  while (scanf("%d %d %d %d %d %d %d", a, a + 1, a + 2, a + 3, a + 4, a + 5, a + 6) == 7) {
    const kv4::Plan p = kv4::plan(a[0], a[1], a[2], a[3], a[4], a[5], a[6]);
    printf("%d %d %d %d\n", p.kind, p.row_tiles, p.chunks, p.chunk_tokens);
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """A function from calls (q_heads, heads, dim, batch, max_q, max_len) to their (kind, row tiles, chunks, tokens a chunk)."""
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(MAIN)
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-I" + os.path.join(ROOT, "bit_quantized_gemm_amd", "csrc"),
                    str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)

    def run(calls):
        text = "\n".join(" ".join(map(str, (*c, 256))) for c in calls)
        out = subprocess.run([str(d / "plan")], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return run


def _calls():
    for heads in (1, 8, 256, 1024):
        for group in (1, 2, 9):
            for dim in (64, 128, 256):
                for batch in (1, 30, 1 << 10, 1 << 15, 1 << 20):
                    for max_q in (1, 9, 17, 130, 1 << 12, 1 << 20):
                        for max_len in (1, 16, 4096, 1 << 20):
                            if group * heads <= 16384 and max_q * group < 1 << 30:
                                yield (group * heads, heads, dim, batch, max_q, max_len)


def test_plans_fit_a_launch(plans):
    """Every call whose prompt tiles are below 2^24 gets a plan below 2^24 workgroups, tiles that hold its rows and chunks
    that hold its tokens; joined rows fit a launch too."""
    calls = list(_calls())
    for (q_heads, heads, dim, batch, max_q, max_len), (kind, tiles, chunks, tokens) in zip(calls, plans(calls)):
        rows, pairs = max_q * q_heads // heads, batch * heads
        what = (q_heads, heads, dim, batch, max_q, max_len, kind, tiles, chunks, tokens)
        if pairs * -(-rows // 128) < 1 << 24:
            assert pairs * tiles * chunks < 1 << 24, what
        assert tiles == -(-rows // (128 if kind == PROMPT else 16)), what
        assert 1 <= chunks <= 64 and (chunks - 1) * tokens < max_len <= chunks * tokens, what
        assert chunks == 1 or pairs * rows < 1 << 24, what


@pytest.mark.parametrize("total_q,q_heads,heads,dim,batch,max_q,max_len", [(1 << 20, 8, 8, 64, 1 << 20, 17, 16),
                                                                            (1 << 20, 512, 256, 64, 1 << 15, 9, 4096)])
def test_calls_below_the_documented_limit_are_accepted(total_q, q_heads, heads, dim, batch, max_q, max_len):
    """2^23 prompt tiles: the faster kernel's 2^24 workgroups of 16 rows would not fit a launch."""
    if not os.path.exists(bq.lib_path()):
        pytest.skip("libatom.so not built (python -m bit_quantized_gemm_amd.build)")
    assert bq.atom_kv4_attention_workspace_bytes(total_q, q_heads, heads, dim, batch, max_q, max_len) >= 0


def test_ranges_reach_every_kernel(plans):
    """The bounds of test_gpu_kv4_range.py: the kernel of 16 rows whole and divided, the kernel of 128 likewise."""
    pytest.importorskip("torch")
    import test_gpu_kv4_range as R
    want = {"decode": (EIGHT, False), "divided": (EIGHT, True), "prompt": (PROMPT, False), "parts": (PROMPT, True)}
    for mode, (total, longest) in R.MODES.items():
        most = max(total, max(R.COUNTS[mode][1]))
        calls = [(4, 2, dim, 2, most, longest // 16 * 16) for dim in (64, 128, 256)]
        for kind, _, chunks, _ in plans(calls):
            assert (kind, chunks > 1) == want[mode], mode


def test_prompt_tests_reach_the_prompt_kernel(plans):
    """test_gpu_kv4_prompt.py, and the two tests of large batches in test_gpu_kv4.py, whole and divided."""
    pytest.importorskip("torch")
    import test_gpu_kv4 as T
    import test_gpu_kv4_prompt as P
    shapes = [(c[0], c[2], c[3], c[4], c[5]) for c in T.CASES]
    shapes += [(lens, Hq, H, D, page) for D in (64, 128, 256) for page in (16, 32, 64) for lens, Hq, H in (
        ([200, 70], 4, 2), ([190, 130], 4, 2), ([73, 50], 2, 1), ([170, 50], 2, 1), ([280, 90], 2, 1))]
    calls = []
    for lens, Hq, H, D, page in shapes:
        total, longest = P.bounds(lens, Hq, H)
        calls.append((Hq, H, D, len(lens), total, min(longest, max(longest // page, -(-max(lens) // page)) * page)))
    calls += [(4 * G, 4, D, 4, 2200, 1100) for D, G in ((128, 2), (64, 3), (64, 1), (128, 4), (256, 2), (256, 3))]
    for c, (kind, _, chunks, _) in zip(calls, plans(calls)):
        assert (kind, chunks) == (PROMPT, 1), c
    calls = [(8, 2, D, 4, 256, 16384) for D in (64, 128, 256)]
    for c, (kind, _, chunks, _) in zip(calls, plans(calls)):
        assert kind == PROMPT and chunks > 1, c


def test_small_batches_take_the_kernel_of_16_rows(plans):
    """The shapes of test_gpu_kv4.py with their own bounds: eight waves up to 16 rows, four beyond."""
    pytest.importorskip("torch")
    import test_gpu_kv4 as T
    calls = [(Hq, H, D, len(lens), max(count), max(lens)) for lens, count, Hq, H, D, _ in T.CASES]
    for c, (kind, _, chunks, _) in zip(calls, plans(calls)):
        assert kind == (EIGHT if c[4] * c[0] // c[1] <= 16 else FOUR) and chunks == 1, c
