"""The KV cache's bookkeeping on the GPU against the CPU oracle (needs an MI355X): whole numbers, so equal."""
import numpy as np
import pytest

from oracle import layer_oracle as O

torch = pytest.importorskip("torch")
import bit_quantized_gemm_amd as bq  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm GPU visible")
    bq.load_library()


def say(*a):
    print(*a, flush=True)


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def state(batch, width, page, longest, seed, spare=20):
    """lens, table, free, state as numpy arrays: sequences in shuffled pages, whatever behind them."""
    r = np.random.default_rng(seed)
    lens = r.integers(0, longest + 1, batch).clip(0, width * page)
    pages = batch * width + spare
    order = r.permutation(pages)
    table = r.integers(-5, pages, (batch, width))
    inside = np.arange(width) < -(-lens // page)[:, None]
    table[inside] = order[:batch * width].reshape(batch, width)[inside]
    free = np.concatenate([order[batch * width:], order[:batch * width][~inside.reshape(-1)]])
    return lens, table, np.concatenate([free, np.full(pages - len(free), -1)]), np.array([len(free), 0])


def check_extend(lens, new, table, free, st, page, total, **k):
    want = O.extend(lens, new, table, free, st, page, total)
    d = [dev(lens), dev(new), dev(table), bq.KV4Pool(dev(free), dev(st))]
    slots, start, out, after = bq.atom_kv4_extend(*d, page, total, **k)
    for a, b in zip((slots, start, out, d[2], after), (want[0], want[1], want[2], want[3], want[4])):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
    np.testing.assert_array_equal(d[0].cpu().numpy(), lens)              # what is no output stays
    np.testing.assert_array_equal(d[3].free.cpu().numpy(), free)
    np.testing.assert_array_equal(d[3].state.cpu().numpy(), st)
    return want


def check_release(done, lens, table, free, st, page):
    want = O.release(done, lens, table, free, st, page)
    d = [dev(done, torch.bool), dev(lens), dev(table), bq.KV4Pool(dev(free), dev(st))]
    out, after = bq.atom_kv4_release(*d, page)
    for a, b in zip((out, d[3].free, after, d[2], d[1]), (*want, table, lens)):
        np.testing.assert_array_equal(a.cpu().numpy(), b)


CASES = [(1, 1, 16, 0, 1), (1, 3, 16, 20, 28), (5, 4, 16, 40, 1), (64, 8, 64, 400, 1), (64, 8, 64, 400, 5), (255, 4, 128, 300, 200),
         (256, 20, 16, 200, 100), (257, 4, 32, 90, 30), (300, 3, 256, 500, 1), (1000, 4, 16, 40, 20), (1024, 3, 16, 40, 1),
         (1025, 3, 16, 40, 1), (1025, 5, 16, 40, 20), (3000, 2, 16, 30, 2), (4, 300, 16, 100, 3000), (2, 200, 256, 5, 20000), (1500, 70, 16, 40, 1000)]


@pytest.mark.parametrize("batch,width,page,longest,most", CASES)
def test_extend(batch, width, page, longest, most):
    say(f"[extend] {batch} x {width} pages of {page}, <= {longest} + {most}")
    r = np.random.default_rng(batch + most)
    lens, table, free, st = state(batch, width, page, longest, 1)
    new = r.integers(0, most + 1, batch)
    exact = max(1, int(new.sum()))
    for total in (exact, exact + 37, max(1, exact // 2)):                # all rows, padded, too few
        check_extend(lens, new, table, free, st, page, total)
    st[0] = max(0, O.extend(lens, new, table, free, st, page, exact)[4][0] * -1 + st[0])      # just enough pages
    assert check_extend(lens, new, table, free, st, page, exact)[4].tolist() == [0, 0]
    if st[0]:
        st[0] -= 1                                                      # one too few: nothing happens
        got = check_extend(lens, new, table, free, st, page, exact)
        assert got[4].tolist() == [st[0], 1] and (got[0] == -1).all()


@pytest.mark.parametrize("batch,width,page,longest,most", CASES)
def test_release(batch, width, page, longest, most):
    say(f"[release] {batch} x {width} pages of {page}, <= {longest}")
    r = np.random.default_rng(batch)
    lens, table, free, st = state(batch, width, page, longest, 2)
    for share in (0.0, 0.3, 1.0):
        check_release(r.random(batch) < share, lens, table, free, st, page)
    st[0] = len(free) - 3                                               # given back twice: what does not fit is dropped
    check_release(np.ones(batch, bool), lens, table, free, st, page)


def test_values_out_of_range():
    """Lengths, counts, states and page ids that no sound state holds: clamped, no fault, nothing else written."""
    lens, table, free, st = state(40, 5, 16, 70, 3)
    lens = np.where(np.arange(40) % 3 == 0, [-5, 1 << 30, -(1 << 31), (1 << 31) - 1] * 10, lens)
    new = np.where(np.arange(40) % 4 == 0, [-1, (1 << 31) - 1, -(1 << 31), 7] * 10, 3)
    free = np.where(np.arange(len(free)) % 5 == 0, -7, free)
    table = np.where(np.arange(5) == 2, -(1 << 31), table)
    for total in (1, 100, 100000):
        for pool in (st[0], 1 << 30, -4, 0, (1 << 31) - 1):
            check_extend(lens, new, table, free, np.array([pool, 9]), 16, total)
            check_release(new > 2, lens, table, free, np.array([pool, 9]), 16)


@pytest.mark.parametrize("batch,total", [(3, 60), (60, 1000), (65, 1030), (300, 900), (700, 9000), (2000, 4000), (2000, 30000)])
def test_in_place(batch, total):
    """Lengths and the pool's state replaced, in one launch or two: the results of a call with outputs of their own."""
    say(f"[pages in place] {batch} sequences, {total} rows")
    lens, table, free, st = state(batch, 20, 16, 150, 4, spare=5000)
    new = np.random.default_rng(5).integers(0, 2 * total // batch, batch)
    want = O.extend(lens, new, table, free, st, 16, total)
    l, t, pool = dev(lens), dev(table), bq.KV4Pool(dev(free), dev(st))
    slots, start, l2, s2 = bq.atom_kv4_extend(l, dev(new), t, pool, 16, total, lens_out=l, state_out=pool.state)
    assert l2 is l and s2 is pool.state
    for a, b in zip((slots, start, l, t, pool.state), want):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
    done = np.arange(batch) % 3 == 0
    lens, free, st = O.release(done, want[2], want[3], free, want[4], 16)
    bq.atom_kv4_release(dev(done, torch.bool), l, t, pool, 16, lens_out=l, state_out=pool.state)
    for a, b in zip((l, pool.free, pool.state), (lens, free, st)):
        np.testing.assert_array_equal(a.cpu().numpy(), b)


def test_a_serving_loop_keeps_its_pages():
    """Steps and releases in turn from a full pool: no page is ever in two places, and all come back."""
    batch, width, page, pages = 20, 12, 16, 150
    r = np.random.default_rng(6)
    pool = bq.kv4_pool(pages)
    lens, table = torch.zeros(batch, dtype=torch.int32, device="cuda"), torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    seen_short = False
    for step in range(60):
        new = r.integers(0, 30, batch)
        l = lens.cpu().numpy()
        new = np.minimum(new, width * page - l)
        bq.atom_kv4_extend(lens, dev(new), table, pool, page, 600, lens_out=lens, state_out=pool.state)
        seen_short |= int(pool.state[1]) > 0
        done = r.random(batch) < 0.25 if step % 3 == 2 else np.zeros(batch, bool)
        bq.atom_kv4_release(dev(done, torch.bool), lens, table, pool, page, lens_out=lens, state_out=pool.state)
        l, t, n = lens.cpu().numpy(), table.cpu().numpy(), int(pool.state[0])
        held = t[np.arange(width) < -(-l // page)[:, None]]
        both = np.concatenate([held, pool.free.cpu().numpy()[:n]])
        assert sorted(both.tolist()) == list(range(pages)), step
    assert seen_short
    bq.atom_kv4_release(torch.ones(batch, dtype=torch.bool, device="cuda"), lens, table, pool, page, lens_out=lens, state_out=pool.state)
    assert pool.state.tolist() == [pages, 0] and not lens.any()


def test_streams_and_graphs():
    lens, table, free, st = state(30, 40, 16, 100, 7)
    l, t, pool = dev(lens), dev(table), bq.KV4Pool(dev(free), dev(st))
    new, done = dev(np.full(30, 3)), torch.zeros(30, dtype=torch.bool, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bq.atom_kv4_extend(l, new, t.clone(), pool, 16, 95, stream=side)
    side.synchronize()
    want = O.extend(lens, np.full(30, 3), table, free, st, 16, 95)
    for a, b in zip(got, (want[0], want[1], want[2], want[4])):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
    graph = torch.cuda.CUDAGraph()
    slots, start = torch.empty(95, dtype=torch.int64, device="cuda"), torch.empty(31, dtype=torch.int32, device="cuda")
    with torch.cuda.graph(graph):
        bq.atom_kv4_release(done, l, t, pool, 16, lens_out=l, state_out=pool.state)
        bq.atom_kv4_extend(l, new, t, pool, 16, 95, slots=slots, q_start=start, lens_out=l, state_out=pool.state)
    for i in range(5):
        d = np.arange(30) % 7 == i
        done.copy_(dev(d, torch.bool))
        n = np.arange(30) % (i + 2)
        new.copy_(dev(n))
        graph.replay()
        torch.cuda.synchronize()
        lens, free, st = O.release(d, lens, table, free, st, 16)
        want = O.extend(lens, n, table, free, st, 16, 95)
        lens, table, st = want[2], want[3], want[4]
        for a, b in zip((slots, start, l, t, pool.state, pool.free), (*want, free)):
            np.testing.assert_array_equal(a.cpu().numpy(), b)


def test_very_many_sequences():
    """More sequences than workgroups have threads many times over: scans of 69 tiles, in several workgroups and in place."""
    batch = 70001
    say(f"[pages] {batch} sequences")
    lens, table, free, st = state(batch, 2, 16, 20, 8)
    new = np.random.default_rng(9).integers(0, 4, batch)
    total = int(new.sum()) + 10
    want = check_extend(lens, new, table, free, st, 16, total)
    l, t, pool = dev(lens), dev(table), bq.KV4Pool(dev(free), dev(st))
    bq.atom_kv4_extend(l, dev(new), t, pool, 16, total, lens_out=l, state_out=pool.state)
    for a, b in zip((l, t, pool.state), (want[2], want[3], want[4])):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
    check_extend(lens, np.where(np.arange(batch) % 1000 == 0, 1, 0), table, free, st, 16, 71)
    check_release(np.arange(batch) % 3 == 0, want[2], want[3], free, want[4], 16)
