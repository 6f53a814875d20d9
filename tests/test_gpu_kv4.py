"""4-bit KV cache on the GPU against the CPU oracle (needs an MI355X): codes, zero points, scales and values
read back bit for bit; attention within a bound derived from its roundings.

Bound of |out - out64| for one query and channel, n tokens in sight, D channels, with w the exact weights (sum 1):
* a score carries the fp32 roundings of a sum of D + 2 products, at most (D + 8) 2^-24 of scale * sum |q| * 15 s
  (codes and zero points are below 16), and of its exponent (|score - max| 2^-22; scores further than 100 below
  weigh nothing): each weight, and the weights' sum, is off by a factor within 1 +- eta;
* a weight times its value scale is rounded to fp16: 2^-11 of it, or half of fp16's smallest step, 2^-25, of at most twice
  the largest value scale u, against a sum of weights of at least 1;
* the sums over tokens are fp32: n 2^-24 of the sum of w * u * (code + zero) <= 30 u, likewise the weights' sum;
* the result's own half step.
So tol = (2^-11 + 2 eta) * sum w |v| + 2^-24 * 15 u^2-free terms (n * 30 u + 2 n * 15 u) + n 2^-24 |out| + eps / 2 |out|.
"""
import numpy as np
import pytest

from oracle import serve_oracle as S

torch = pytest.importorskip("torch")
import bit_quantized_gemm_amd as bq  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm GPU visible")
    bq.load_library()


def say(*a):
    print(*a, flush=True)


def f32(t):
    return t.detach().float().cpu().numpy()


def randn(*shape, seed, dtype=torch.float16, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * gain).to(dtype).cuda()


def garbage(pages, page, H, D, seed=0):
    """A cache whose every byte is arbitrary: parameters are infinities and NaN among others."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = bq.kv4_cache(pages, page, H, D)
    for t in c:
        t.view(torch.uint8).copy_(torch.randint(0, 256, t.view(torch.uint8).shape, generator=g, device="cuda", dtype=torch.uint8))
    return c


def host(cache):
    return [t.cpu().numpy().copy() for t in cache]


def same(cache, want):
    for t, w in zip(cache, want):
        np.testing.assert_array_equal(t.cpu().numpy().view(np.uint8), w.view(np.uint8))


# ------------------------------------------------------------------ append and read
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,D,page,tokens", [(1, 64, 16, 1), (2, 128, 16, 5), (3, 256, 32, 40), (8, 128, 64, 70),
                                             (5, 64, 128, 33), (2, 128, 256, 3), (32, 128, 64, 9)])
def test_append_and_read(H, D, page, tokens, dtype):
    say(f"[kv4 append] H={H} D={D} page={page} tokens={tokens} {dtype}")
    t = TYPES[dtype]
    pages = tokens // page + 3
    cache = garbage(pages, page, H, D)
    K, V = randn(tokens, H, D, seed=1, dtype=t), randn(tokens, H, D, seed=2, dtype=t, gain=0.1)
    K[0, 0] = 0                                          # nothing but zeros
    V[-1, -1] = 3                                        # a constant
    if tokens > 2:
        K[1, 0] = K[1, 0].abs()                          # one sign only
        V[1, 0] = -V[1, 0].abs()
        K[2, 0, :4] = 60000                              # far out
        V[2, 0] *= 1e-6                                  # next to fp16's smallest scale
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(3))[:tokens].cuda()
    if tokens > 4:
        slots[3], slots[4] = -1, pages * page            # outside the cache: skipped
    want = host(cache)
    for side, x in enumerate((K, V)):
        S.kv4_write(want, page, slots.tolist(), side, *S.kv4_quantize(f32(x)))
    bq.atom_kv4_append(K, V, slots, cache)
    same(cache, want)                                    # the bytes of every other token as they were
    rk, rv = bq.atom_kv4_read(cache, slots, dtype=t)
    for side, r in enumerate((rk, rv)):
        exact = torch.from_numpy(S.kv4_read(want, page, slots.tolist(), side))
        assert torch.equal(r.cpu(), exact.to(t)), side


def test_append_borders():
    """Quotients on and next to borders between codes, over scales of fp16's whole range, in both types."""
    for t in TYPES.values():
        rows = []
        for a in (15.0, 7.5, 1.0, 0.1, 1000.0, 3e-4, 65000.0):
            for z in range(0, 16, 3):
                s = np.float32(np.float16(a / 15))
                x = torch.tensor([-(z * s), (15 - z) * s] + [float((k + 0.5 - z) * s) for k in range(15)] * 2).to(t)
                x = torch.cat([x, (x.view(torch.int16) + 1).view(t), (x.view(torch.int16) - 1).view(t)])
                rows.append(torch.cat([x, torch.zeros(128 - x.numel(), dtype=t)]).clamp(-(z * s), float((15 - z) * s)))
        x = torch.stack(rows).nan_to_num(0, 0, 0).view(-1, 1, 128).cuda()
        n = x.shape[0]
        cache = bq.kv4_cache(n // 16 + 1, 16, 1, 128)
        want = host(cache)
        slots = torch.arange(n, device="cuda")
        for side in (0, 1):
            S.kv4_write(want, 16, slots.tolist(), side, *S.kv4_quantize(f32(x)))
        bq.atom_kv4_append(x, x, slots, cache)
        same(cache, want)


def test_append_huge_values():
    x = torch.full((1, 1, 64), 1e38, dtype=torch.bfloat16, device="cuda")
    x[0, 0, ::2] = -3e38
    cache = bq.kv4_cache(1, 16, 1, 64)
    bq.atom_kv4_append(x, x, torch.zeros(1, dtype=torch.int64, device="cuda"), cache)
    want = host(bq.kv4_cache(1, 16, 1, 64))
    for side in (0, 1):
        S.kv4_write(want, 16, [0], side, *S.kv4_quantize(f32(x)))
    same(cache, want)


def test_append_rows_apart_and_streams():
    qkv = randn(20, 3 * 2 * 64, seed=4)
    K, V = qkv[:, 128:256].view(20, 2, 64), qkv[:, 256:].view(20, 2, 64)
    slots = torch.arange(20, device="cuda") + 5
    a, b = bq.kv4_cache(2, 16, 2, 64), bq.kv4_cache(2, 16, 2, 64)
    bq.atom_kv4_append(K, V, slots, a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bq.atom_kv4_append(K.contiguous(), V.contiguous(), slots, b, stream=side)
    rk, rv = bq.atom_kv4_read(b, slots, stream=side)
    side.synchronize()
    same(a, host(b))
    for x, y in zip((rk, rv), bq.atom_kv4_read(a, slots)):
        assert torch.equal(x, y)


def test_cache_past_32_bits():
    """More than 2^32 bytes of codes a side: tokens of the last page land there and nowhere else."""
    pages, page, H, D = 9000, 64, 128, 128
    cache = bq.KV4Cache(*(torch.empty(s, dtype=t, device="cuda") for s, t in (
        ((pages, H, page, D // 2), torch.uint8), ((pages, H, page, 2), torch.float16),
        ((pages, H, page // 4, D // 4, 8), torch.uint8), ((pages, H, page, 2), torch.float16))))
    assert cache.k.numel() > 1 << 32
    small = bq.kv4_cache(2, page, H, D)
    tokens = 100
    K, V = randn(tokens, H, D, seed=5), randn(tokens, H, D, seed=6)
    far = torch.arange(tokens, device="cuda") + (pages - 2) * page
    bq.atom_kv4_append(K, V, far, cache)
    bq.atom_kv4_append(K, V, far - (pages - 2) * page, small)
    for a, b in zip(bq.atom_kv4_read(cache, far), bq.atom_kv4_read(small, far - (pages - 2) * page)):
        assert torch.equal(a, b)
    q = randn(1, H, D, seed=7)
    table = torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([tokens], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    a = bq.atom_kv4_attention(q, cache, table, lens, start)
    b = bq.atom_kv4_attention(q, small, table - (pages - 2), lens, start)
    assert torch.equal(a, b)


# ------------------------------------------------------------------ attention
class Batch:
    """Sequences of `lens` tokens, the last `count` of them queries, in shuffled pages of a pool that holds garbage
    everywhere else."""

    def __init__(self, lens, count, Hq, H, D, page, dtype=torch.float16, seed=0, q_gain=1.0, k_gain=1.0, v_gain=1.0,
                 spare_rows=0, stretch=0):
        self.lens, self.count, self.page = lens, count, page
        width = max(1, -(-max(lens) // page)) + stretch
        pages = len(lens) * width + 1
        g = torch.Generator().manual_seed(seed)
        self.table = torch.randperm(pages, generator=g)[:len(lens) * width].view(len(lens), width).int().cuda()
        self.cache = garbage(pages, page, H, D, seed)
        for i, n in enumerate(lens):
            if n:
                t = torch.arange(n, device="cuda")
                slots = self.table[i].long()[t // page] * page + t % page
                bq.atom_kv4_append(randn(n, H, D, seed=seed + 10 * i + 1, gain=k_gain),
                                   randn(n, H, D, seed=seed + 10 * i + 2, gain=v_gain), slots, self.cache)
        total = sum(count)
        self.total = total
        self.q = randn(total + spare_rows, Hq, D, seed=seed + 5, dtype=dtype, gain=q_gain)
        at = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
        self.start, self.len_t = torch.from_numpy(at).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")

    def run(self, **k):
        return bq.atom_kv4_attention(k.pop("q", self.q), self.cache, self.table, self.len_t, self.start, **k)

    def check(self, out, scale=None, what=""):
        D, Hq = self.q.shape[2], self.q.shape[1]
        scale = D ** -0.5 if scale is None else scale
        cache, q, got, first = host(self.cache), f32(self.q).astype(np.float64), f32(out).astype(np.float64), 0
        H = cache[0].shape[1]
        eps = torch.finfo(out.dtype).eps / 2
        for i, (n, c) in enumerate(zip(self.lens, self.count)):
            t = np.arange(n)
            slots = self.table[i].cpu().numpy().astype(np.int64)[t // self.page] * self.page + t % self.page
            key, value = S.kv4_read(cache, self.page, slots, 0), S.kv4_read(cache, self.page, slots, 1)
            qi = q[first:first + c]
            want, mag, _ = S.attention(qi, key, value, scale)
            p, r = slots // self.page, slots % self.page
            s = np.repeat(cache[1][p, :, r, 1].astype(np.float64).max(0, initial=0), Hq // H)      # [Hq]
            u = np.repeat(cache[3][p, :, r, 1].astype(np.float64).max(0, initial=0), Hq // H)
            eta = (D + 8) * 2.0**-24 * scale * np.abs(qi).sum(2) * 15 * s + 100 * 2.0**-22          # [c, Hq]
            tol = ((2.0**-11 + 2 * eta)[..., None] * mag + 2.0**-24 * n * 60 * u[None, :, None]
                   + (n * 2.0**-24 + eps) * np.abs(want) + 2.0**-25)
            err = np.abs(got[first:first + c] - want)
            assert np.all(err <= tol), (f"{what} sequence {i} ({n} tokens, {c} queries): worst {np.max(err / tol):.3g} of the "
                                        f"bound, error {err.max():.3g} at {np.unravel_index((err / tol).argmax(), err.shape)}")
            first += c


# (lens, count, Hq, H, D, page): lengths around the kernels' units of 16, 32, 64, 128 tokens; every group size; one
# query, a few, and more rows than a tile
CASES = [
    ([1], [1], 1, 1, 64, 16),
    ([1, 2, 15, 16, 17], [1] * 5, 4, 2, 128, 16),
    ([31, 32, 33, 63, 64, 65], [1] * 6, 8, 1, 128, 32),
    ([127, 128, 129, 255, 257, 700], [1] * 6, 5, 5, 64, 64),
    ([130, 513], [1, 1], 16, 2, 256, 128),
    ([1000, 3], [1, 1], 16, 1, 128, 256),
    ([50, 0, 7, 300], [1, 1, 0, 1], 6, 2, 128, 16),          # an empty sequence, and one without queries
    ([5, 40], [8, 3], 4, 4, 64, 16),                         # more queries than tokens: the first see nothing
    ([100, 33, 64], [5, 2, 3], 8, 2, 128, 16),               # 20 rows: two tiles of 16
    ([200, 90], [4, 7], 8, 2, 256, 64),
    ([300, 41], [5, 5], 64, 8, 128, 32),                     # 40 rows
    ([77, 129], [77, 60], 4, 2, 64, 16),                     # prompts
    ([150, 64, 1], [150, 33, 1], 3, 1, 128, 64),
    ([140], [140], 2, 2, 256, 16),
    ([333, 0, 20], [70, 4, 20], 10, 2, 128, 32),
    ([90], [3], 71, 1, 64, 64),                              # a group that divides no tile
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case, dtype):
    lens, count, Hq, H, D, page = CASES[case]
    say(f"[kv4 attention] lens={lens} q={count} heads={Hq}/{H} D={D} page={page} {dtype}")
    b = Batch(lens, count, Hq, H, D, page, TYPES[dtype], seed=case, spare_rows=2)
    out = torch.full_like(b.q, 7.0)
    assert b.run(out=out, max_q=max(count), max_len=max(lens)) is out
    b.check(out)
    assert torch.all(out[b.total:] == 7)                     # rows behind the last sequence
    again = torch.full_like(out, 7.0)
    b.run(out=again, max_q=max(count), max_len=max(lens))
    assert torch.equal(out, again)                           # no order to depend on
    b.check(b.run())                                         # the bounds that Q and the table give
    b.check(b.run(workspace=torch.empty(0, dtype=torch.uint8, device="cuda")), what="undivided")


@pytest.mark.parametrize("q,Hq,H,D", [(1, 8, 8, 128), (1, 32, 4, 64), (3, 8, 1, 128), (20, 8, 4, 128), (40, 2, 1, 256)])
def test_long_sequences_divided(q, Hq, H, D):
    """Lengths that are divided into many chunks, ragged, with a chunk that only some rows see."""
    lens = [5000, 1030, 129, 4097]
    count = [q, max(1, q - 1), 1, q]
    say(f"[kv4 divided] q={q} heads={Hq}/{H} D={D}")
    b = Batch(lens, count, Hq, H, D, 64, seed=q, stretch=2)
    need = bq.atom_kv4_attention_workspace_bytes(sum(count), Hq, H, D, len(lens), q, 5000)
    assert need > 0
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")       # NaN: contents must not matter
    out = b.run(max_q=q, max_len=5000, workspace=ws)
    b.check(out)
    assert torch.all(ws[need:] == 0xFF)
    assert torch.equal(out, b.run(max_q=q, max_len=5000))
    b.check(b.run(), what="bounds from the table")


@pytest.mark.parametrize("lens,count,Hq,H,D", [([15000, 400], [20, 20], 32, 4, 128), ([16000, 900, 12], [100, 33, 12], 4, 1, 64),
                                               ([16384, 5000], [1, 1], 8, 1, 64), ([16384], [40], 32, 1, 128),
                                               ([9000, 16000], [2, 1], 2, 1, 256)])
def test_many_chunks(lens, count, Hq, H, D):
    """Divided 10 to 64 ways: joined by one wave a row in several batches, and by four."""
    say(f"[kv4 many chunks] {lens} {count} heads={Hq}/{H} D={D}")
    b = Batch(lens, count, Hq, H, D, 64, seed=D)
    assert bq.atom_kv4_attention_workspace_bytes(sum(count), Hq, H, D, len(lens), max(count), 16384) >= 10 * sum(count) * Hq * D * 4
    out = b.run(max_q=max(count), max_len=16384)
    b.check(out)
    assert torch.equal(out, b.run(max_q=max(count), max_len=16384))


@pytest.mark.parametrize("k", [dict(q_gain=60.0), dict(q_gain=1e-4), dict(v_gain=1e-4), dict(v_gain=300.0), dict(k_gain=1e-3),
                               dict(k_gain=40.0, q_gain=0.02), dict(scale=3.0), dict(scale=1e-3)])
@pytest.mark.parametrize("q", [1, 30])
def test_attention_magnitudes(q, k):
    """Scores far apart and all alike, values next to fp16's ends."""
    k = dict(k)
    scale = k.pop("scale", None)
    say(f"[kv4 magnitudes] q={q} {k} scale={scale}")
    b = Batch([200, 70], [q, q], 4, 2, 128, 16, seed=3, **k)
    b.check(b.run(scale=scale), scale=scale)


def test_attention_scales_that_rise_and_fall():
    """Value scales that grow by powers of ten along the sequence, and fall again: the weights' common exponent is
    raised on the way.  The bound's u is the largest scale, so the small values in front are held to it."""
    for q in (1, 40):
        b = Batch([400], [q], 2, 1, 128, 16, seed=9)
        t = torch.arange(400, device="cuda")
        slots = b.table[0].long()[t // 16] * 16 + t % 16
        g = 10.0 ** (4 - (t.float() - 200).abs() / 40)
        bq.atom_kv4_append(randn(400, 1, 128, seed=1), (randn(400, 1, 128, seed=2).float() * g[:, None, None]).half(), slots, b.cache)
        b.check(b.run())
        zero = torch.zeros(400, 1, 128, dtype=torch.float16, device="cuda")
        bq.atom_kv4_append(randn(400, 1, 128, seed=1), zero, slots, b.cache)
        assert not b.run().any()                             # values that are all zero (scales of zero)
        bq.atom_kv4_append(zero, randn(400, 1, 128, seed=2), slots, b.cache)
        b.check(b.run())                                     # keys that are all zero: the mean


def test_attention_of_zero_and_non_finite_queries():
    """A zero query weighs all tokens alike; one that holds an infinity or NaN spoils its own row only."""
    for q in (4, 40):
        b = Batch([90, 100], [q, q], 4, 2, 64, 16, seed=5)
        b.q[1] = 0
        out = b.run()
        b.check(out)
        b.q[2, 1, 3], b.q[q, 0, 0] = float("nan"), float("inf")
        bad = b.run()
        for r, h in ((2, 1), (q, 0)):
            assert not bad[r, h].isfinite().any()
            bad[r, h] = out[r, h]
        assert torch.equal(bad, out)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q", [3, 40, 100])
def test_tokens_behind_a_query_do_not_touch_it(q, D):
    """The last two tokens are huge, infinite or NaN: only the queries that see them may notice.  The others keep their
    result up to the weights' rounding to fp16, whose unit is set by the value scales that they see themselves.  Both runs
    round each weight once (2^-12 of it) and the result once (2^-12 of it, or 2^-25): together at most 2^-11 of the largest
    |value| and 2^-11 of the result; values of standard deviation 1e-3 stay below 6e-3, and the bound has twice that."""
    n = 70 + q
    for page in (16, 64):
        b = Batch([n, 50], [q, min(q, 50)], 2, 1, D, page, seed=11, v_gain=1e-3)
        plain = b.run()
        b.check(plain)
        at = torch.arange(n - 2, n, device="cuda")
        slots = b.table[0].long()[at // page] * page + at % page
        before = plain[:q - 2].clone()
        for fill in (60000.0, float("inf"), -float("inf"), float("nan")):
            say(f"[kv4 behind] q={q} D={D} page={page} {fill}")
            x = torch.full((2, 1, D), fill, dtype=torch.float16, device="cuda")
            x[1, 0, ::2] = 1.0
            bq.atom_kv4_append(x, x, slots, b.cache)
            got = b.run()
            assert torch.equal(got[q:], plain[q:])           # the other sequence
            torch.testing.assert_close(got[:q - 2], before, rtol=2.0**-10, atol=2.0**-10 * 6e-3)


def test_attention_strided_queries_and_tight_bounds():
    b = Batch([100, 60, 30], [6, 4, 2], 4, 2, 128, 16, seed=6)
    wide = torch.zeros(b.total, 3 * 4 * 128, dtype=torch.float16, device="cuda")
    wide[:, 512:1024] = b.q.view(b.total, -1)
    out = b.run()
    assert torch.equal(b.run(q=wide[:, 512:1024].view(b.total, 4, 128)), out)
    # queries behind max_q are left as they were; the others still count as the last of their sequence
    some = b.run(max_q=4, out=torch.full_like(out, 7.0))
    keep = torch.tensor([0, 1, 2, 3, 6, 7, 8, 9, 10, 11])
    torch.testing.assert_close(some[keep], out[keep], rtol=2e-3, atol=2e-3)
    assert torch.all(some[4:6] == 7)
    # lengths behind max_len are taken as max_len
    b.lens = [64, 60, 30]
    b.check(b.run(max_len=64))


def test_bad_tables_lengths_and_starts_do_not_fault():
    """Entries outside their ranges are clamped: garbage in their own sequences, the others right.  (The clamps are
    walked over on the host in test_oracle_serve.py.)"""
    for q in (1, 20):
        b = Batch([100, 60, 90], [q, q, q], 4, 2, 64, 16, seed=7)
        out = b.run()
        b.table[1, 0], b.table[1, 1] = -5, 1 << 30
        got = b.run()
        assert torch.equal(got[:q], out[:q]) and torch.equal(got[2 * q:], out[2 * q:])
        b.len_t[1] = 1 << 30
        got = b.run()
        assert torch.equal(got[:q], out[:q]) and torch.equal(got[2 * q:], out[2 * q:])
        b.len_t[1] = -3
        got = b.run()
        assert torch.equal(got[:q], out[:q]) and not got[q:2 * q].any()
        b.start[3] = 1 << 30
        b.run(out=torch.full_like(out, 7.0))
        b.start[1] = -9
        b.run(out=torch.full_like(out, 7.0))
        torch.cuda.synchronize()


def test_two_calls_at_once_on_two_streams():
    a, b = Batch([3000, 900], [1, 1], 8, 2, 128, 64, seed=1), Batch([2500, 1700], [1, 1], 8, 2, 128, 64, seed=2)
    want = a.run(), b.run()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for x in (s, t):
        x.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        got.append((a.run(stream=s), b.run(stream=t)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, want[0]) and torch.equal(y, want[1])


# Bounds far above what the sequences hold choose the launch of a large batch: many query rows in workgroups of 128 (which
# small batches do not take), whole, or divided against a context of up to 16384 tokens.
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page,D,G", [(16, 128, 2), (32, 64, 3), (64, 64, 1), (64, 128, 4), (128, 256, 2), (16, 256, 3)])
def test_prompts_in_a_large_batch(page, D, G, dtype):
    lens, count = [300, 129, 0, 97], [150, 129, 4, 1]
    say(f"[kv4 prompts] page={page} D={D} G={G} {dtype}")
    b = Batch(lens, count, 4 * G, 4, D, page, TYPES[dtype], seed=page + G, spare_rows=2200 - sum(count), stretch=800 // page)
    assert bq.atom_kv4_attention_workspace_bytes(2200, 4 * G, 4, D, 4, 2200, 1100) == 0
    out = torch.full_like(b.q, 7.0)
    b.run(out=out, max_len=1100)
    b.check(out)
    assert torch.all(out[b.total:] == 7)
    again = torch.full_like(out, 7.0)
    b.run(out=again, max_len=1100)
    assert torch.equal(out, again)
    # a row of zeros, one that holds a NaN, and tokens behind the queries that are huge: none touches another row
    b.q[1], b.q[3, 0, 0] = 0, float("nan")
    at = torch.arange(299, 300, device="cuda")
    slots = b.table[0].long()[at // page] * page + at % page
    x = torch.full((1, 4, D), float("inf"), dtype=torch.float16, device="cuda")
    bq.atom_kv4_append(x, x, slots, b.cache)
    got = b.run(out=torch.full_like(out, 7.0), max_len=1100)
    assert not got[3, 0].isfinite().any()
    got[3, 0] = out[3, 0]
    keep = [r for r in range(b.total) if r not in (1, 149)]
    # each weight is rounded once on either side (2^-12 of it), the result once (eps / 2): values are below 6
    torch.testing.assert_close(got[keep], out[keep], rtol=2 * torch.finfo(out.dtype).eps, atol=2.0**-11 * 6)


@pytest.mark.parametrize("page,D,dtype", [(16, 128, "bf16"), (32, 64, "fp16"), (128, 256, "fp16"), (64, 128, "fp16")])
def test_prompt_parts_against_long_contexts(page, D, dtype):
    """A part of a prompt against a long context, divided among workgroups, with pages that end inside a tile, sequences
    shorter than the others and one without tokens."""
    say(f"[kv4 prompt part] page={page} D={D}")
    count = [70, 66, 5, 1]
    b = Batch([4200, 130, 0, 700], count, 8, 2, D, page, TYPES[dtype], seed=page, spare_rows=256 - sum(count),
              stretch=(16384 - 4200) // page)
    assert bq.atom_kv4_attention_workspace_bytes(256, 8, 2, D, 4, 256, 16384) > 0
    out = torch.full_like(b.q, 7.0)
    b.run(out=out, max_len=16384)
    b.check(out)
    assert torch.all(out[b.total:] == 7)
    b.check(b.run(max_len=16384, workspace=torch.empty(0, dtype=torch.uint8, device="cuda")), what="undivided")
    b.check(b.run(max_q=70, max_len=4200), what="tight bounds")


def test_shared_and_repeated_pages():
    """Two sequences whose tables name the same pages (a common prefix), one of them the same page twice."""
    b = Batch([64, 48, 60], [1, 1, 1], 4, 2, 64, 16, seed=13)
    b.table[1] = b.table[0]
    b.table[2, 1] = b.table[2, 0]
    b.check(b.run())
    b.check(b.run(max_q=1, max_len=64))


def test_two_graphs_of_divided_sequences():
    """Two captured graphs and eager calls in turn, on streams of their own: each call has its own workspace."""
    bs = [Batch([3000, 900], [1, 1], 8, 2, 128, 64, seed=1), Batch([2500, 1700], [40, 3], 8, 2, 128, 64, seed=2)]
    for b in bs:
        b.run()
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g, b in zip(graphs, bs):
        with torch.cuda.graph(g):
            outs.append(b.run())
    for i in range(4):
        for b in bs:
            b.q.copy_(randn(*b.q.shape, seed=50 + i))
        for g in graphs:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        eager = [b.run() for b in bs]
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            assert torch.equal(o, e)
    for b, o in zip(bs, outs):
        b.check(o)


# ------------------------------------------------------------------ a layer as it would be used
def _layer(Hq, H, D, hidden, dtype):
    W = [bq.atom_quantize_w8a8(randn(n, k, seed=20 + i, dtype=dtype, gain=k ** -0.5))
         for i, (n, k) in enumerate([((Hq + 2 * H) * D, hidden), (hidden, Hq * D)])]

    def step(x, cache, slots, table, lens, start, **k):
        qkv = bq.linear_w8a8(x, *W[0])
        n = x.shape[0]
        q, key, value = (t.view(n, -1, D) for t in qkv.split([Hq * D, H * D, H * D], 1))
        bq.atom_kv4_append(key, value, slots, cache)
        o = bq.atom_kv4_attention(q, cache, table, lens, start, **k)
        return qkv, o, bq.linear_w8a8(o.view(n, -1), *W[1])
    return step, W


@pytest.mark.parametrize("dtype", TYPES)
def test_layer_prompt_then_decode(dtype):
    """Projection, append, attention and output projection over a ragged prompt batch, then decode steps, the last of
    them captured once and replayed: the tokens' own queries, keys and values against the oracle at each step."""
    t = TYPES[dtype]
    Hq, H, D, hidden, page = 4, 2, 64, 200, 16
    step, W = _layer(Hq, H, D, hidden, t)
    lens, width = [20, 37], 5
    table = torch.randperm(2 * width, generator=torch.Generator().manual_seed(1)).view(2, width).int().cuda()
    cache = garbage(2 * width, page, H, D)
    b = Batch.__new__(Batch)
    b.cache, b.table, b.page = cache, table, page

    def slots_of(i, pos):
        return int(table[i, pos // page]) * page + pos % page

    def verify(qkv, o, y, now, count):
        b.lens, b.count = list(now), list(count)
        n = qkv.shape[0]
        b.q = qkv[:, :Hq * D].reshape(n, Hq, D)
        b.check(o)
        want, _ = S.gemm_w8a8(*S.quantize_w8a8(f32(o.reshape(n, -1))), W[1][0].cpu().numpy(), W[1][1].cpu().numpy())
        np.testing.assert_allclose(f32(y), want, rtol=torch.finfo(t).eps, atol=1e-5)

    x = randn(sum(lens), hidden, seed=30, dtype=t)
    slots = torch.tensor([slots_of(i, p) for i in range(2) for p in range(lens[i])], device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    verify(*step(x, cache, slots, table, torch.tensor(lens, **i32), torch.tensor([0, lens[0], sum(lens)], **i32)), lens, lens)

    start, now = torch.tensor([0, 1, 2], **i32), torch.tensor(lens, **i32)
    x, slots = torch.zeros(2, hidden, dtype=t, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")

    def feed(k):
        for i in range(2):
            lens[i] += 1
            slots[i] = slots_of(i, lens[i] - 1)
        now.copy_(torch.tensor(lens, **i32))
        x.copy_(randn(2, hidden, seed=40 + k, dtype=t))

    feed(0)
    verify(*step(x, cache, slots, table, now, start, max_q=1), lens, [1, 1])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    feed(1)
    with torch.cuda.graph(graph):
        out = step(x, cache, slots, table, now, start, max_q=1)
    for k in range(2, 7):
        graph.replay()
        torch.cuda.synchronize()
        verify(*out, lens, [1, 1])
        feed(k)                                              # the program's own eager work between replays
