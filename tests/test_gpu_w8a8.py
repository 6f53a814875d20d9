"""W8A8 layer on the GPU against the CPU oracle (needs an MI355X): codes and scales bit for bit, Y within
its fp32 steps and one rounding of the exact value.

Bound of |Y - y64|: the product acc * sx * sw takes three fp32 roundings (the integer's conversion, the scale
product, the fma), each at most 2^-24 of |acc sx sw| or of |y|, then Y's own half step, eps / 2 of |y|
(2^-25 for fp16's smallest numbers).
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
    """A 16-bit float tensor's values on the host."""
    return t.detach().float().cpu().numpy()


def make(rows, K, dtype, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g) * gain
    x[:, torch.randint(0, K, (max(1, K // 100),), generator=g)] *= 20
    return x.to(dtype).cuda()


def check_y(Y, y64, mag, what):
    y = f32(Y).astype(np.float64)
    eps = torch.finfo(Y.dtype).eps / 2
    assert np.abs(y64).max() < 6e4
    tol = eps * np.abs(y64) * (1 + 2.0**-20) + 2.0**-24 * (3 * mag + np.abs(y64)) + (2.0**-25 if Y.dtype == torch.float16 else 0)
    err = np.abs(y - y64)
    assert np.all(err <= tol), f"{what}: worst {np.max(err - tol):.3g} over, at {np.unravel_index((err - tol).argmax(), err.shape)}"


def check_codes(Xq, sx, x):
    q, s = S.quantize_w8a8(f32(x))
    np.testing.assert_array_equal(sx.cpu().numpy().view(np.uint32), s.view(np.uint32))
    np.testing.assert_array_equal(Xq.cpu().numpy(), q)
    return q, s


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 7), (5, 64), (4, 128), (9, 129), (2, 512), (7, 520), (6, 2048), (5, 2049),
                                    (3, 4096), (3, 4097), (2, 8192), (2, 11008), (3, 16384), (2, 16385), (2, 65536),
                                    (1, 65535), (385, 520), (390, 1155), (400, 2048), (1025, 8192), (1026, 5001)])
def test_quantize(rows, K, dtype):
    say(f"[w8a8 quantize] {rows}x{K} {dtype}")
    x = make(rows, K, TYPES[dtype], rows + K)
    Xq, sx = bq.atom_quantize_w8a8(x, Xq=torch.full((rows, bq.atom_w8a8_row_bytes(K)), 99, dtype=torch.int8, device="cuda"))
    check_codes(Xq, sx, x)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_borders(dtype):
    """Values that lie on or next to a border between two codes: x = max (k + 1/2) / 127 rounded to the
    type, its neighbours, halves of the maximum; maxima over the type's whole range; zero rows."""
    t = TYPES[dtype]
    rows = []
    for a in [1.0, 1.5, 127.0, 254.0, 0.37, 60000.0, 6.1e-5, 3e-7, 2.0**-24] + ([1e-30, 1e-38, 2.0**-133, 1e38] if dtype == "bf16" else []):
        a = torch.tensor(a).to(t).float().item()
        x = torch.cat([torch.tensor([a]), a * (torch.arange(-127, 127) + 0.5) / 127, a * torch.arange(-64, 64) / 128]).to(t)
        bits = x.view(torch.int16)
        rows.append(torch.cat([x, (bits + 1).view(t), (bits - 1).view(t)]).nan_to_num(0, 0, 0).clamp(-a, a))
    rows.append(torch.zeros_like(rows[0]))
    x = torch.stack([r[:1100] for r in rows]).to(t).cuda()
    x = torch.where(x.isfinite(), x, 0.0)
    check_codes(*bq.atom_quantize_w8a8(x), x)


def test_quantize_rows_apart_and_shifted():
    wide = make(12, 1000, torch.float16, 5)
    for x in (wide[:, :512], wide[:, 8:520], wide[:, 1:514], wide[::3, 3:700], wide[2:3, 5:]):
        check_codes(*bq.atom_quantize_w8a8(x), x)


def test_quantize_survives_inf_and_nan():
    """No fault, and the rows beside them are right."""
    x = make(6, 300, torch.float16, 6)
    x[1, 3], x[4, 299] = float("inf"), float("nan")
    Xq, sx = bq.atom_quantize_w8a8(x)
    keep = [0, 2, 3, 5]
    check_codes(Xq[keep], sx[keep], x[keep])


# every kind of kernel and its edges: few rows (one and two tiles), divided K, the three tile sizes
SHAPES = [(1, 1, 1), (1, 17, 300), (1, 4096, 4096), (3, 130, 127), (16, 100, 11008), (17, 33, 1000), (32, 1000, 513),
          (33, 64, 128), (33, 65, 4096), (33, 65, 6145), (127, 1000, 5000), (300, 300, 300), (4000, 31, 1000), (64, 128, 2048), (65, 127, 4100), (100, 260, 65536), (128, 4096, 1024),
          (333, 777, 1155), (257, 4097, 300), (512, 8192, 256), (1024, 4100, 384), (4000, 4104, 200), (2304, 11008, 130)]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K, dtype, bias):
    say(f"[w8a8 linear] {M}x{N}x{K} {dtype} bias={bias}")
    t = TYPES[dtype]
    x, w = make(M, K, t, M + K), make(N, K, t, N + K + 1, 0.02)
    b = make(1, N, t, 3)[0] if bias else None
    Wq, sw = bq.atom_quantize_w8a8(w)
    Y = bq.linear_w8a8(x, Wq, sw, bias=b)
    Xq, sx = bq.atom_quantize_w8a8(x)
    acc = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    acc.addmm_(Xq.double(), Wq.double().t())        # integers below 2^53
    p = acc * sx.double()[:, None] * sw.double()
    y64 = (p + b.double() if bias else p).cpu().numpy()
    check_y(Y, y64, p.abs().cpu().numpy(), f"{M}x{N}x{K}")
    if M * N * K < 3e8:                             # the oracle's own product, from its own codes
        want, _ = S.gemm_w8a8(*check_codes(Xq, sx, x), *check_codes(Wq, sw, w), None if b is None else f32(b))
        np.testing.assert_allclose(y64, want, rtol=1e-12, atol=1e-9)
    need = bq.atom_gemm_w8a8_workspace_bytes(M, N, K)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda") if need else None
    for work in (ws, None):                         # divided or not: the same bits
        torch.testing.assert_close(bq.atom_gemm_w8a8(Xq, sx, Wq, sw, K, bias=b, dtype=t, workspace=work), Y, rtol=0, atol=0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(1, 33, 16384), (2, 20, 8192), (3, 48, 5461), (4, 65, 4096), (4, 16, 4097), (1, 70, 16385), (2, 5, 1),
                                   (4, 1, 129), (3, 4096, 513)])
def test_up_to_four_tokens_equal_two_steps(M, N, K, dtype):
    """Quantized and multiplied in one launch, at the ends of what that takes: the bits of the two steps, also from rows
    that lie apart and start at odd elements."""
    say(f"[w8a8 one launch] {M}x{N}x{K} {dtype}")
    t = TYPES[dtype]
    Wq, sw = bq.atom_quantize_w8a8(make(N, K, t, 1, 0.02))
    wide = make(M, K + 9, t, 2)
    wide[M - 1, 3:] = 0                              # a row of zeros
    wide[0, K // 2] = 1000                           # and one with an outlier
    for first in (0, 1, 3, 8):
        x = wide[:, first:first + K]
        Y = bq.linear_w8a8(x, Wq, sw)
        torch.testing.assert_close(Y, bq.atom_gemm_w8a8(*bq.atom_quantize_w8a8(x), Wq, sw, K, dtype=t), rtol=0, atol=0)
        torch.testing.assert_close(Y, bq.linear_w8a8(x.contiguous(), Wq, sw), rtol=0, atol=0)
        ws = torch.empty(bq.atom_linear_w8a8_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
        torch.testing.assert_close(Y, bq.linear_w8a8(x, Wq, sw, Y=torch.empty_like(Y), workspace=ws), rtol=0, atol=0)
    keep = wide.clone()
    odd = torch.full((M, K + 9), float("nan"), dtype=t, device="cuda")       # what lies around the rows is not read into them
    odd[:, 5:5 + K] = keep[:, 5:5 + K]
    torch.testing.assert_close(bq.linear_w8a8(odd[:, 5:5 + K], Wq, sw), bq.linear_w8a8(keep[:, 5:5 + K].contiguous(), Wq, sw),
                               rtol=0, atol=0)


def test_two_graphs_and_eager_calls_between():
    """Two captured graphs of the same shapes and eager calls in turn: none reads another's workspace."""
    for M, N, K in ((2, 300, 1000), (64, 128, 4096), (64, 128, 8192)):
        Wq, sw = bq.atom_quantize_w8a8(make(N, K, torch.float16, 1, 0.02))
        xs = [make(M, K, torch.float16, 2 + i) for i in range(2)]
        bq.linear_w8a8(xs[0], Wq, sw)
        torch.cuda.synchronize()
        graphs, ys = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
        for g, x in zip(graphs, xs):
            with torch.cuda.graph(g):
                ys.append(bq.linear_w8a8(x, Wq, sw))
        for i in range(4):
            for x in xs:
                x.copy_(make(M, K, torch.float16, 20 + i + x.data_ptr() % 7))
            streams = torch.cuda.Stream(), torch.cuda.Stream()
            for g, s in zip(graphs, streams):
                s.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(s):
                    g.replay()
            eager = [bq.linear_w8a8(x, Wq, sw) for x in xs]
            torch.cuda.synchronize()
            for y, e, x in zip(ys, eager, xs):
                torch.testing.assert_close(y, e, rtol=0, atol=0)


def test_extreme_sums():
    """The largest sums: every code +-127 over the longest K, exactly -+127^2 * 65536."""
    K = bq.MAX_K
    for M, N in ((5, 40), (40, 40), (300, 200)):
        Xq = torch.full((M, K), 127, dtype=torch.int8, device="cuda")
        Wq = torch.full((N, K), -127, dtype=torch.int8, device="cuda")
        Wq[0] = 127
        one = torch.full((max(M, N),), 2.0**-15, device="cuda")
        Y = bq.atom_gemm_w8a8(Xq, one[:M].contiguous(), Wq, one[:N].contiguous(), K)
        want = torch.full((M, N), -(127.0**2) * 2.0**-14, device="cuda")
        want[:, 0] *= -1
        torch.testing.assert_close(Y, want.half(), rtol=0, atol=0)


def test_few_rows_equal_many_rows():
    """A token's result does not depend on the batch it comes in."""
    x, w = make(300, 1000, torch.bfloat16, 1), make(500, 1000, torch.bfloat16, 2)
    Wq, sw = bq.atom_quantize_w8a8(w)
    Y = bq.linear_w8a8(x, Wq, sw)
    for n in (1, 16, 17, 32, 33, 64, 200):
        torch.testing.assert_close(bq.linear_w8a8(x[:n], Wq, sw), Y[:n], rtol=0, atol=0)


def test_given_buffers_and_streams():
    x, w = make(40, 700, torch.float16, 1), make(90, 700, torch.float16, 2)
    Wq, sw = bq.atom_quantize_w8a8(w)
    want = bq.linear_w8a8(x, Wq, sw)
    Y = torch.full((42, 90), 7.0, dtype=torch.float16, device="cuda")
    ws = torch.empty(bq.atom_linear_w8a8_workspace_bytes(40, 90, 700), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert bq.linear_w8a8(x, Wq, sw, Y=Y[:40], workspace=ws, stream=side) is not None
    side.synchronize()
    torch.testing.assert_close(Y[:40], want, rtol=0, atol=0)
    assert torch.all(Y[40:] == 7)                   # rows behind the last are left as they were
    with torch.cuda.stream(side):
        again = bq.linear_w8a8(x, Wq, sw)
    other = bq.linear_w8a8(x, Wq, sw, stream=side)
    side.synchronize()
    torch.testing.assert_close(again, want, rtol=0, atol=0)
    torch.testing.assert_close(other, want, rtol=0, atol=0)


@pytest.mark.parametrize("M,N,K", [(1, 512, 1024), (20, 300, 500), (64, 128, 4096), (64, 128, 8192), (300, 1000, 640)])
def test_graph_replays(M, N, K):
    say(f"[w8a8 graph] {M}x{N}x{K}")
    x, w = make(M, K, torch.float16, 1), make(N, K, torch.float16, 2, 0.02)
    Wq, sw = bq.atom_quantize_w8a8(w)
    bq.linear_w8a8(x, Wq, sw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = bq.linear_w8a8(x, Wq, sw)
    for i in range(4):
        x.copy_(make(M, K, torch.float16, 10 + i))
        graph.replay()
        torch.cuda.synchronize()
        torch.testing.assert_close(Y, bq.linear_w8a8(x, Wq, sw), rtol=0, atol=0)


def test_output_past_32_bits():
    """More than 2^32 bytes of Y: the last rows against a small product of their own."""
    M, N, K = 140000, 16384, 64
    say(f"[w8a8 large] {M}x{N}x{K}")
    x, w = make(M, K, torch.float16, 1), make(N, K, torch.float16, 2, 0.02)
    Wq, sw = bq.atom_quantize_w8a8(w)
    Y = bq.linear_w8a8(x, Wq, sw)
    for rows in (slice(0, 40), slice(70000, 70040), slice(M - 40, M)):
        torch.testing.assert_close(Y[rows], bq.linear_w8a8(x[rows], Wq, sw), rtol=0, atol=0)


def test_quantize_more_rows_than_a_launch():
    """2^24 rows of 2049 elements (69 GB): 256 threads each are 2^32, one more than a launch takes.  Zero rows but a few."""
    rows, K = 1 << 24, 2049
    rb = bq.atom_w8a8_row_bytes(K)
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < rows * (2 * K + rb) + (8 << 30):
        pytest.skip("needs 114 GB of device memory")
    say(f"[w8a8 quantize] {rows}x{K}")
    try:
        x = torch.zeros(rows, K, dtype=torch.float16, device="cuda")
        Xq, sx = torch.full((rows, rb), 0x55, dtype=torch.int8, device="cuda"), torch.full((rows,), -1.0, device="cuda")
        at = torch.tensor([0, 5, (1 << 23) + 1, rows - 257, rows - 2, rows - 1], device="cuda")
        x[at] = make(len(at), K, torch.float16, 7)
        bq.atom_quantize_w8a8(x, Xq=Xq, sx=sx)
        check_codes(Xq[at], sx[at], x[at])
        Xq[at], sx[at] = 0, 0
        assert not sx.any()
        assert all(not part.view(torch.int64).any() for part in Xq.split(1 << 20))
    finally:
        x = Xq = sx = None
        torch.cuda.empty_cache()
