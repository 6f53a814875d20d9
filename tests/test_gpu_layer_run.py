"""A decoder layer's attention block as a server runs it on these operators (needs an MI355X): tokens admitted (pages, slots,
table), the norm with quantized rows, a quantized projection, keys and values appended to the 4-bit cache, attention over it,
and pages given back; eager and as a captured step, for the W8A8 and the MXFP4 layer.  And the refusals of the new calls
with tensors on the device."""
import numpy as np
import pytest

from oracle import layer_oracle as O

torch = pytest.importorskip("torch")
import bit_quantized_gemm_amd as bq  # noqa: E402

pytestmark = pytest.mark.gpu
HEADS, KV, DIM, PAGE, WIDTH = 8, 2, 64, 16, 6
HIDDEN = HEADS * DIM


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm GPU visible")
    bq.load_library()


def say(*a):
    print(*a, flush=True)


class Layer:
    """Weights and state of one layer for `batch` sequences."""

    def __init__(self, kind, batch, seed):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.batch = kind, batch
        self.norm_w = (1 + 0.2 * torch.randn(HIDDEN, generator=g)).half().cuda()
        w = (torch.randn((HEADS + 2 * KV) * DIM, HIDDEN, generator=g) * 0.05).half().cuda()
        o = (torch.randn(HIDDEN, HIDDEN, generator=g) * 0.05).half().cuda()
        pack = bq.atom_quantize_mxfp4 if kind == "mx" else bq.atom_quantize_w8a8
        self.qkv, self.out = pack(w), pack(o)
        self.cache = bq.kv4_cache(batch * WIDTH, PAGE, KV, DIM)
        self.pool = bq.kv4_pool(batch * WIDTH)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.table = torch.zeros((batch, WIDTH), dtype=torch.int32, device="cuda")

    def step(self, x, residual, new, total):
        """One pass over `total` rows, new[b] of them for sequence b; lengths, table and pool are replaced."""
        slots, start, _, _ = bq.atom_kv4_extend(self.lens, new, self.table, self.pool, PAGE, total, lens_out=self.lens,
                                                state_out=self.pool.state)
        norm = bq.atom_rmsnorm_mxfp4 if self.kind == "mx" else bq.atom_rmsnorm_w8a8
        gemm = bq.atom_gemm_mxfp4 if self.kind == "mx" else bq.atom_gemm_w8a8
        linear = bq.linear_mxfp4 if self.kind == "mx" else bq.linear_w8a8
        xq, sx, h = norm(x, self.norm_w, 1e-5, residual=residual)
        qkv = gemm(xq, sx, *self.qkv, HIDDEN, dtype=x.dtype).view(total, HEADS + 2 * KV, DIM)
        q, k, v = qkv.split((HEADS, KV, KV), 1)
        bq.atom_kv4_append(k, v, slots, self.cache)
        out = torch.zeros((total, HEADS, DIM), dtype=x.dtype, device="cuda")
        bq.atom_kv4_attention(q, self.cache, self.table, self.lens, start, max_q=total, out=out)
        return linear(out.view(total, HIDDEN), *self.out), h, slots, out

    def finish(self, done):
        bq.atom_kv4_release(done, self.lens, self.table, self.pool, PAGE, lens_out=self.lens, state_out=self.pool.state)


def inputs(total, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(total, HIDDEN, generator=g).half().cuda() for _ in range(2))


def reference(layer, history, x, residual, new):
    """Attention's output of the same step in fp64 from the operators' definitions, and how far the kernels' may be from it;
    `history`: each sequence's keys and values as the cache holds them.

    A query is a projection's fp16 output: off by 2^-11 of itself, and by the sum's own steps, K / 64 instructions of four
    additions of 2^-23 of sum |x w| = mag.  So a score is off by at most ds, weights by a factor of e^(2 ds) and their mean of the
    values by (e^(2 ds) - 1) of the largest; attention's weights and output are fp16: 2^-9 of the largest value more."""
    def weights(t):
        if layer.kind == "mx":
            return O.mx_values(*O.mx_unpack(t[0].cpu().numpy(), t[1].cpu().numpy()))[:, :HIDDEN]
        return t[0][:, :HIDDEN].cpu().numpy().astype(np.float64) * t[1].cpu().numpy().astype(np.float64)[:, None]

    def quantized(y):
        if layer.kind == "mx":
            return O.mx_values(*O.mx_codes(y))[:, :HIDDEN]
        q, s = O.w8_codes(y)
        return q[:, :HIDDEN] * s.astype(np.float64)[:, None]
    f16 = lambda a: a.astype(np.float16).astype(np.float32)  # noqa: E731
    y, _ = O.rmsnorm(x.float().cpu().numpy(), layer.norm_w.float().cpu().numpy(), 1e-5, residual.float().cpu().numpy(), f16)
    y, w = quantized(y), weights(layer.qkv)
    qkv = (y @ w.T).reshape(len(x), -1, DIM)
    off = np.abs(qkv) * 2.0**-11 + (np.abs(y) @ np.abs(w).T).reshape(qkv.shape) * (HIDDEN / 64 * 4 * 2.0**-23)
    out, bound, row = np.zeros((len(x), HEADS, DIM)), np.zeros((len(x), HEADS, 1)), 0
    for b, n in enumerate(new):
        for i in range(n):
            for j in range(HEADS):
                keys, values = (t[:len(t) - n + i + 1, j // (HEADS // KV)] for t in history[b])
                s = keys @ qkv[row, j] / np.sqrt(DIM)
                p = np.exp(s - s.max())
                out[row, j] = (p / p.sum()) @ values
                ds = (np.abs(keys) @ off[row, j]).max() / np.sqrt(DIM)
                bound[row, j] = (np.expm1(2 * ds) + 2.0**-9) * np.abs(values).max()
            row += 1
    return out, bound


@pytest.mark.parametrize("kind", ["w8", "mx"])
def test_a_step_is_its_parts(kind):
    """Prompts, then single tokens (some sequences take none): sums, lengths and slots as they have to be, attention's output
    against fp64, and the last projection's that of the same rows."""
    batch = 5
    layer = Layer(kind, batch, 1)
    lens = np.zeros(batch, int)
    for step, new in enumerate(([3, 20, 1, 17, 40], [1] * 5, [1, 0, 2, 0, 1], [1] * 5)):
        total = sum(new) + 3
        x, r = inputs(total, step)
        y, h, slots, out = layer.step(x, r, torch.tensor(new, dtype=torch.int32, device="cuda"), total)
        torch.testing.assert_close(h, x + r, rtol=0, atol=0)
        lens += new
        assert layer.lens.tolist() == lens.tolist() and (slots[-3:] == -1).all()
        history, table = [], layer.table.cpu().numpy()
        for b in range(batch):
            at = torch.tensor([int(table[b, t // PAGE]) * PAGE + t % PAGE for t in range(lens[b])], device="cuda", dtype=torch.int64)
            history.append(tuple(t.double().cpu().numpy() for t in bq.atom_kv4_read(layer.cache, at)))
        rows = sum(new)
        want, bound = reference(layer, history, x[:rows], r[:rows], new)
        err = np.abs(out[:rows].double().cpu().numpy() - want)
        assert (err <= bound).all(), (step, float((err - bound).max()))
        assert not out[rows:].any()                     # rows behind the last sequence are left as they were
        linear = bq.linear_mxfp4 if kind == "mx" else bq.linear_w8a8
        torch.testing.assert_close(y, linear(out.view(total, HIDDEN).clone(), *layer.out), rtol=0, atol=0)
    done = torch.tensor([True, False, True, False, False], device="cuda")
    layer.finish(done)
    assert layer.lens.tolist() == [0, lens[1], 0, lens[3], lens[4]]


@pytest.mark.parametrize("kind", ["w8", "mx"])
def test_a_captured_step(kind):
    """The whole step and the release in a graph, replayed with new inputs and eager work in between, against the same steps
    run eagerly on a second layer."""
    say(f"[layer graph] {kind}")
    batch, total = 4, 12
    a, b = Layer(kind, batch, 2), Layer(kind, batch, 2)
    x, r = inputs(total, 0)
    new, done = torch.zeros(batch, dtype=torch.int32, device="cuda"), torch.zeros(batch, dtype=torch.bool, device="cuda")
    a.step(x, r, new, total)                            # (no tokens: state as it was)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h, slots, _ = a.step(x, r, new, total)
        a.finish(done)
    for i in range(6):
        x2, r2 = inputs(total, 10 + i)
        x.copy_(x2)
        r.copy_(r2)
        new.copy_(torch.tensor([3, 1, (i * 5) % 7, 1]))
        done.copy_(torch.tensor([False, i == 3, False, i == 4]))
        graph.replay()
        want = b.step(x, r, new, total)
        b.finish(done)
        torch.cuda.synchronize()
        rows = int(new.sum())
        for got, ref in zip((y[:rows], h, slots), (want[0][:rows], want[1], want[2])):
            torch.testing.assert_close(got, ref, rtol=0, atol=0)
        for got, ref in zip((a.lens, a.table, *a.pool), (b.lens, b.table, *b.pool)):
            torch.testing.assert_close(got, ref, rtol=0, atol=0)


def z(*shape, dtype=torch.float16, device="cuda"):
    return torch.zeros(shape, dtype=dtype, device=device)


def test_refusals_on_the_device():
    """What is not well-formed ends in an AtomError whatever path a call takes.  No call here launches."""
    u8, i8, i32, f32 = torch.uint8, torch.int8, torch.int32, torch.float32
    X, W, Wq, sw = z(4, 300), z(300), z(6, 256, dtype=u8), z(2, 6, 8, dtype=u8)
    Xq, sx, Q8, s8 = z(4, 256, dtype=u8), z(2, 4, 8, dtype=u8), z(4, 384, dtype=i8), z(4, dtype=f32)
    lens, table, pool, done = z(5, dtype=i32), z(5, 3, dtype=i32), bq.kv4_pool(9), z(5, dtype=torch.bool)
    ext = dict(lens=lens, new=lens.clone(), table=table, pool=pool, page=16, total=7)
    rel = dict(done=done, lens=lens, table=table, pool=pool, page=16)
    calls = [
        *(lambda a=a: bq.linear_mxfp4(*a) for a in (
            (z(), Wq, sw), (X[0], Wq, sw), (z(0, 300), Wq, sw), (z(4, 0), Wq, sw), (X, Wq[:, :150], sw), (X, Wq[0], sw), (X, Wq, sw[:1]),
            (X, Wq, sw[:, :5]), (X, Wq, z()), (X, Wq, sw, z()), (X, Wq, sw, z(6).bfloat16()), (X.float(), Wq, sw), (X, Wq.cpu(), sw),
            (X, Wq, sw.cpu()), (X[:1].expand(4, 300), Wq, sw), (z(300, 4).t(), Wq, sw), (X, Wq.view(i8), sw), (X, Wq, sw, None, z(4, 5)),
            (X, Wq, sw, None, None, z()), (z(9, 8000), z(6, 4096, dtype=u8), z(32, 6, 8, dtype=u8), None, None, z(8, dtype=u8)))),
        *(lambda a=a: bq.atom_quantize_mxfp4(*a) for a in ((z(),), (X[0],), (z(0, 300),), (X.float(),), (z(300, 4).t(),), (X, z(4, 150, dtype=u8)),
                                                           (X, None, z(2, 3, 8, dtype=u8)), (X[:, ::2],), (X[:1].expand(4, 300),))),
        *(lambda a=a: bq.atom_dequantize_mxfp4(*a) for a in ((Xq, sx, 0), (Xq, sx, 600), (Xq, sx, 200), (Xq, sx[:1], 300), (Xq.view(i8), sx, 300),
                                                             (Xq, sx, 300, f32), (Xq.cpu(), sx, 300), (z(0, 256, dtype=u8), z(2, 0, 8, dtype=u8), 300))),
        *(lambda a=a: bq.atom_dequantize_w8a8(*a) for a in ((Q8, s8, 0), (Q8, s8, 385), (Q8, s8, 200), (Q8, s8[:3], 300), (Q8.view(u8), s8, 300),
                                                            (Q8, s8, 300, f32), (Q8, s8.half(), 300), (Q8, s8.cpu(), 300))),
        *(lambda a=a: bq.atom_gemm_mxfp4(*a) for a in ((Xq, sx, Wq, sw, 600), (Xq, sx[:1], Wq, sw, 300), (Xq, sx, Wq[:, :128], sw, 300),
                                                       (Xq, sx, Wq, sw, 300, z(5)), (Xq, sx, Wq, sw, 300, None, z(4, 5)),
                                                       (Xq, sx, Wq, sw, 300, z(6).bfloat16(), None, torch.float16),
                                                       (Xq, sx, Wq, sw, 300, None, None, f32), (Xq, sx, Wq.cpu(), sw, 300),
                                                       (Xq, sx, Wq, sw, 300, None, None, None, z(9)),
                                                       (Xq, sx, Wq, sw, 300, None, None, None, z(4, 4, dtype=u8)))),
        *(lambda f=f, k=k: f(**{**dict(X=X, weight=W), **k}) for f in (bq.atom_rmsnorm_w8a8, bq.atom_rmsnorm_mxfp4) for k in (
            dict(X=z()), dict(X=X[0]), dict(X=z(0, 300)), dict(X=X.float()), dict(X=X[:, ::2]), dict(X=z(300, 4).t()), dict(weight=W[:299]),
            dict(weight=W.bfloat16()), dict(weight=W.cpu()), dict(weight=z(600)[::2]), dict(residual=X[:3]), dict(residual=X.bfloat16()),
            dict(residual=X.cpu()), dict(residual=z(300, 4).t()), dict(residual=z(1, 300).expand(4, 300)), dict(eps=0.0), dict(eps=-1.0),
            dict(eps=float("nan")), dict(eps=float("inf")), dict(H=X), dict(residual=X, H=z(4, 299)), dict(residual=X, H=W), dict(Xq=Xq[:3]),
            dict(sx=s8[:3]), dict(residual=z(4, 300), H=X[:, :299]), dict(residual=z(3, 300)))),
        *(lambda k=k: bq.atom_kv4_extend(**{**ext, **k}) for k in (
            dict(lens=lens[:4]), dict(lens=lens.long()), dict(lens=lens.cpu()), dict(new=lens[:4]), dict(new=lens.float()), dict(table=table[0]),
            dict(table=table.long()), dict(table=z(3, 5, dtype=i32).t()), dict(table=z(0, 3, dtype=i32), lens=lens[:0], new=lens[:0]),
            dict(table=z(5, 0, dtype=i32)), dict(pool=None), dict(pool=pool[:1]), dict(pool=pool._replace(free=table)),
            dict(pool=pool._replace(free=z(0, dtype=i32))), dict(pool=pool._replace(state=z(3, dtype=i32))), dict(pool=pool._replace(state=z(2))),
            dict(page=0), dict(page=24), dict(page=8), dict(page=512), dict(page=-16), dict(total=0), dict(total=-5), dict(total=(1 << 24) + 1),
            dict(slots=z(7, dtype=i32)), dict(slots=z(8, dtype=torch.int64)), dict(q_start=z(5, dtype=i32)), dict(lens_out=z(4, dtype=i32)),
            dict(lens_out=table[0:1].view(-1)), dict(lens_out=ext["new"]), dict(state_out=pool.free[:2]), dict(lens=table.view(-1)[:5]),
            dict(table=pool.free[:5].view(5, 1)))),
        *(lambda k=k: bq.atom_kv4_release(**{**rel, **k}) for k in (
            dict(done=done[:4]), dict(done=done.to(u8)), dict(done=done.cpu()), dict(lens=lens[:4]), dict(lens=lens.long()), dict(table=table[0]),
            dict(table=table.cpu()), dict(pool=None), dict(pool=pool._replace(free=table)), dict(pool=pool._replace(state=lens)), dict(page=20),
            dict(lens_out=table.view(-1)[:5]), dict(state_out=lens[:2], lens_out=lens), dict(lens_out=pool.free[:5]))),
    ]
    for i, call in enumerate(calls):
        print(i, flush=True)
        with pytest.raises(bq.AtomError):
            call()


def calls(t=torch.float16):
    """Each new operator's call on well-formed tensors, as a function of a stream (None: the short way)."""
    g = torch.Generator().manual_seed(3)
    X, W = torch.randn(9, 700, generator=g).to(t).cuda(), torch.randn(700, generator=g).to(t).cuda()
    Wq, sw = bq.atom_quantize_mxfp4(torch.randn(50, 700, generator=g).to(t).cuda())
    b = torch.randn(50, generator=g).to(t).cuda()
    q4, q8 = bq.atom_quantize_mxfp4(X), bq.atom_quantize_w8a8(X)
    lens = torch.tensor([3, 40, 0, 17], dtype=torch.int32, device="cuda")
    new, done = torch.tensor([5, 1, 2, 30], dtype=torch.int32, device="cuda"), torch.tensor([True, False, True, True], device="cuda")
    table, pool = torch.arange(16, dtype=torch.int32, device="cuda").view(4, 4), bq.kv4_pool(30)
    return [lambda s: bq.linear_mxfp4(X, Wq, sw, stream=s), lambda s: bq.linear_mxfp4(X[:2], Wq, sw, b, stream=s),
            lambda s: bq.linear_mxfp4(X[::2], Wq, sw, b, stream=s), lambda s: bq.atom_quantize_mxfp4(X, stream=s),
            lambda s: bq.atom_gemm_mxfp4(*q4, Wq, sw, 700, dtype=t, stream=s), lambda s: bq.atom_gemm_mxfp4(*q4, Wq, sw, 700, b, stream=s),
            lambda s: bq.atom_gemm_mxfp4(*q4, Wq, sw, 700, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"), stream=s),
            lambda s: bq.atom_dequantize_mxfp4(*q4, 700, dtype=t, stream=s), lambda s: bq.atom_dequantize_w8a8(*q8, 700, dtype=t, stream=s),
            *(lambda s, f=f, r=r: f(X, W, 1e-5, residual=r, stream=s) for f in (bq.atom_rmsnorm_w8a8, bq.atom_rmsnorm_mxfp4)
              for r in (None, X.flip(0).contiguous())),
            lambda s: bq.atom_kv4_extend(lens, new, table, pool, 16, 41, stream=s),
            lambda s: bq.atom_kv4_release(done, lens, table, pool, 16, stream=s)]


def flat(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_short_and_full_way_agree(dtype):
    """The extension module and the full checks call the same kernels: the same outputs, types and shapes; neither keeps a reference
    or memory.  (The extension module is built with the library.)"""
    import sys
    assert bq._SHORT is not None
    for i, call in enumerate(calls(dtype)):
        print(i, flush=True)
        short, full = flat(call(None)), flat(call(torch.cuda.current_stream()))
        keep = bq._SHORT
        bq._SHORT = None
        try:
            without = flat(call(None))
        finally:
            bq._SHORT = keep
        assert len(short) == len(full) == len(without)
        for a, b, c in zip(short, full, without):
            assert a.dtype == b.dtype == c.dtype and a.shape == b.shape == c.shape and a.is_contiguous() and not a.requires_grad
            torch.testing.assert_close(a, b, rtol=0, atol=0)
            torch.testing.assert_close(a, c, rtol=0, atol=0)
        del short, full, without, a, b, c
        call(None)
        torch.cuda.synchronize()
        used, none = torch.cuda.memory_allocated(), sys.getrefcount(None)
        for _ in range(500):
            call(None)
        torch.cuda.synchronize()
        assert torch.cuda.memory_allocated() == used and abs(sys.getrefcount(None) - none) < 100


def test_short_way_takes_the_current_stream():
    """Work queued on a side stream in front of a call there is seen by it."""
    side = torch.cuda.Stream()
    X = torch.zeros(64, 4096, dtype=torch.float16, device="cuda")
    Wq, sw = bq.atom_quantize_mxfp4(torch.ones(32, 4096, dtype=torch.float16, device="cuda"))
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(5):
            big = big @ big * 1e-3
        X.fill_(1.0)
        Y = bq.linear_mxfp4(X, Wq, sw)
    side.synchronize()
    torch.testing.assert_close(Y, torch.full_like(Y, 4096.0), rtol=0, atol=0)
