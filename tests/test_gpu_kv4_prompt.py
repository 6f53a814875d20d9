"""The kernel of 128 query rows on the shapes, magnitudes and bad neighbours that small batches bring to the kernel of 16 (needs an
MI355X): the same calls with bounds of a large batch, which select it (pinned in test_kv4_plan.py).  Bounds of the errors:
test_gpu_kv4.py."""
import pytest

from test_gpu_kv4 import CASES, TYPES, Batch, randn, say

torch = pytest.importorskip("torch")
import bit_quantized_gemm_amd as bq  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm GPU visible")
    bq.load_library()


def bounds(lens, Hq, H):
    """Rows of Q and longest context that the launch is planned for: 70000 rows of all sequences and kv heads."""
    return -(-70000 // (Hq * len(lens))), 300 if max(lens) <= 288 else 1100


def batch(lens, count, Hq, H, D, page=16, **k):
    total, longest = bounds(lens, Hq, H)
    assert total >= sum(count)
    b = Batch(lens, count, Hq, H, D, page, spare_rows=total - sum(count), stretch=max(0, longest // page - -(-max(lens) // page)), **k)
    b.run_it = lambda **a: b.run(max_len=longest, **a)
    return b


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case, dtype):
    lens, count, Hq, H, D, page = CASES[case]
    say(f"[kv4 prompt kernel] lens={lens} q={count} heads={Hq}/{H} D={D} page={page} {dtype}")
    b = batch(lens, count, Hq, H, D, page, dtype=TYPES[dtype], seed=case)
    out = torch.full_like(b.q, 7.0)
    b.run_it(out=out)
    b.check(out)
    assert torch.all(out[b.total:] == 7)
    again = torch.full_like(b.q, 7.0)
    b.run_it(out=again)
    assert torch.equal(out, again)


MAGNITUDES = [dict(q_gain=60.0), dict(q_gain=1e-4), dict(v_gain=1e-4), dict(v_gain=300.0), dict(k_gain=1e-3),
              dict(k_gain=40.0, q_gain=0.02), dict(scale=3.0), dict(scale=1e-3)]


@pytest.mark.parametrize("k", MAGNITUDES)
@pytest.mark.parametrize("D,page", [(64, 64), (128, 16), (128, 64), (256, 32)])
def test_magnitudes(D, page, k):
    k = dict(k)
    scale = k.pop("scale", None)
    say(f"[kv4 prompt kernel] magnitudes D={D} page={page} {k} scale={scale}")
    b = batch([200, 70], [90, 40], 4, 2, D, page, seed=3, **k)
    b.check(b.run_it(scale=scale), scale=scale)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_zero_and_non_finite_queries(page, D):
    b = batch([190, 130], [60, 40], 4, 2, D, page, seed=5)
    b.q[1] = 0
    out = b.run_it()
    b.check(out)
    b.q[2, 1, 3], b.q[60, 0, 0] = float("nan"), float("inf")
    bad = b.run_it()
    for r, h in ((2, 1), (60, 0)):
        assert not bad[r, h].isfinite().any()
        bad[r, h] = out[r, h]
    assert torch.equal(bad[:b.total], out[:b.total])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q", [3, 100])
def test_tokens_behind_a_query_do_not_touch_it(q, D):
    """As in test_gpu_kv4.py, which derives the bound: the last two tokens are huge, infinite or NaN."""
    n = 70 + q
    for page in (16, 64):
        b = batch([n, 50], [q, min(q, 50)], 2, 1, D, page, seed=11, v_gain=1e-3)
        plain = b.run_it()
        b.check(plain)
        at = torch.arange(n - 2, n, device="cuda")
        slots = b.table[0].long()[at // page] * page + at % page
        for fill in (60000.0, float("inf"), -float("inf"), float("nan")):
            say(f"[kv4 prompt kernel] behind q={q} D={D} page={page} {fill}")
            x = torch.full((2, 1, D), fill, dtype=torch.float16, device="cuda")
            x[1, 0, ::2] = 1.0
            bq.atom_kv4_append(x, x, slots, b.cache)
            got = b.run_it()
            assert torch.equal(got[q:b.total], plain[q:b.total])
            torch.testing.assert_close(got[:q - 2], plain[:q - 2], rtol=2.0**-10, atol=2.0**-10 * 6e-3)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_value_scales_that_rise_and_fall(D):
    """Scales by powers of ten up and down along the sequence; values all zero; keys all zero (the mean)."""
    b = batch([280, 90], [120, 30], 2, 1, D, seed=9)
    t = torch.arange(280, device="cuda")
    slots = b.table[0].long()[t // 16] * 16 + t % 16
    g = 10.0 ** (4 - (t.float() - 140).abs() / 28)
    bq.atom_kv4_append(randn(280, 1, D, seed=1), (randn(280, 1, D, seed=2).float() * g[:, None, None]).half(), slots, b.cache)
    b.check(b.run_it())
    zero = torch.zeros(280, 1, D, dtype=torch.float16, device="cuda")
    bq.atom_kv4_append(randn(280, 1, D, seed=1), zero, slots, b.cache)
    assert not b.run_it()[:120].any()
    bq.atom_kv4_append(zero, randn(280, 1, D, seed=2), slots, b.cache)
    b.check(b.run_it())
