"""MXFP4 layer on the GPU against the CPU oracle (needs an MI355X): codes and scales bit for bit, Y exactly where every step
of the sum is exact in fp32, else within the sum's steps and one rounding.

Bound of |Y - y64|: an instruction adds its blocks' sums (two of 32, or four) to the accumulator: at most four additions of fp32,
each off by at most 2^-23 (a truncation) of the magnitudes so far, at most mag = sum |x w|; there are K / 64 instructions, then at
most 16 waves' or 4 pieces' sums and the bias, 2^-24 each; then Y's own half step, eps / 2 of |y| (2^-25 for fp16's
smallest numbers).
"""
import numpy as np
import pytest

from oracle import layer_oracle as O

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


def make(rows, K, dtype, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g) * gain
    x[:, torch.randint(0, K, (max(1, K // 100),), generator=g)] *= 20
    return x.to(dtype).cuda()


def check_codes(Xq, sx, x):
    c, s = O.mx_codes(f32(x))
    q, s3 = O.mx_pack(c, s)
    np.testing.assert_array_equal(sx.cpu().numpy(), s3)
    np.testing.assert_array_equal(Xq.cpu().numpy(), q)
    return c, s


def values(q, s):
    """fp64 values [rows, padded K] of packed rows, on the device."""
    grid = torch.tensor(O.GRID, device="cuda")
    grid = torch.cat([grid, -grid])
    v = grid[torch.stack([q & 15, q >> 4], -1).long()].flatten(1)
    e = s.permute(1, 0, 2).flatten(1).double() - 127
    return v * torch.exp2(e).repeat_interleave(32, 1)


def check_y(Y, x, w, bias, K, what):
    y = x @ w.t().contiguous()
    mag = x.abs() @ w.abs().t().contiguous()
    if bias is not None:
        y, mag = y + bias.double(), mag + bias.double().abs()
    eps = torch.finfo(Y.dtype).eps / 2
    tol = eps * y.abs() * (1 + 2.0**-10) + (K / 64 * 4 * 2.0**-23 + 20 * 2.0**-24) * mag + (2.0**-25 if Y.dtype == torch.float16 else 0)
    over = (Y.double() - y).abs() - tol
    assert float(y.abs().max()) < 6e4
    assert bool((over <= 0).all()), f"{what}: worst {float(over.max()):.3g} over"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 7), (5, 31), (4, 32), (9, 33), (2, 255), (7, 256), (17, 257), (16, 520), (15, 2048),
                                    (5, 2049), (33, 4096), (2, 11008), (1, 65535), (2, 65536), (385, 1155), (11003, 1155), (8203, 2056)])
def test_quantize_and_back(rows, K, dtype):
    say(f"[mxfp4 quantize] {rows}x{K} {dtype}")
    t = TYPES[dtype]
    x = make(rows, K, t, rows + K)
    rb, g = bq.atom_mxfp4_row_bytes(K), bq.atom_mxfp4_groups(K)
    u8 = dict(dtype=torch.uint8, device="cuda")
    Xq, sx = bq.atom_quantize_mxfp4(x, Xq=torch.full((rows, rb), 99, **u8), sx=torch.full((g, rows, 8), 99, **u8))
    c, s = check_codes(Xq, sx, x)
    back = bq.atom_dequantize_mxfp4(Xq, sx, K, dtype=t)
    want = torch.from_numpy(O.mx_values(c, s)[:, :K]).float().to(t)
    torch.testing.assert_close(back.cpu(), want, rtol=0, atol=0)


@pytest.mark.parametrize("dtype", TYPES)
def test_every_value_and_border(dtype):
    """Every finite value of the type as a block's largest and beside a larger one: borders, neighbours, subnormal numbers."""
    t = TYPES[dtype]
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(t)
    x = torch.where(x.isfinite(), x, 0.0)
    top = x.float().abs()
    rows = [x.repeat_interleave(32).view(-1, 4096)]                       # blocks of one value
    for gain in (1.0, 1.25, 1.4):                                         # sorted: each block's values are near its largest
        rows.append((torch.sort(top).values * gain).clamp(max=torch.finfo(t).max).to(t).view(-1, 4096))
    g = torch.Generator().manual_seed(1)
    rows.append(x[torch.randperm(1 << 16, generator=g)].view(-1, 4096))
    # borders of the eight codes for maxima of every exponent
    border = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0])
    lo, hi = (-26, 12) if dtype == "fp16" else (-133, 124)
    b = torch.cat([(border * 2.0**e).to(t) for e in range(lo, hi)])
    b = torch.cat([b, -b]).view(-1, 16)
    near = (b.view(torch.int16) + 1).view(t)
    under = torch.where(b == 0, b, (b.view(torch.int16) - 1).view(t))
    blocks = torch.cat([torch.cat([b, near], 1), torch.cat([b, under], 1)])
    blocks = torch.where(blocks.isfinite(), blocks, 0.0)
    rows.append(torch.cat([blocks.flatten(), torch.zeros(-blocks.numel() % 4096, dtype=t)]).view(-1, 4096))
    x = torch.cat(rows).cuda()
    check_codes(*bq.atom_quantize_mxfp4(x), x)


def test_rows_apart_and_shifted():
    wide = make(40, 1000, torch.float16, 5)
    for x in (wide[:, :512], wide[:, 8:520], wide[:, 1:514], wide[::3, 3:700], wide[2:3, 5:]):
        check_codes(*bq.atom_quantize_mxfp4(x), x)
    around = torch.full_like(wide, float("nan"))                          # what lies around the rows is not read into them
    around[:, 5:600] = wide[:, 5:600]
    check_codes(*bq.atom_quantize_mxfp4(around[:, 5:600]), wide[:, 5:600])


@pytest.mark.parametrize("dtype", TYPES)
def test_inf_and_nan(dtype):
    """A block with an inf or NaN has the scale NaN, the blocks beside it their own; Y's row is NaN, the others are right."""
    t = TYPES[dtype]
    x = make(6, 600, t, 6)
    x[1, 3], x[4, 599], x[4, 40], x[2, 100] = float("inf"), float("nan"), -float("inf"), 0
    Xq, sx = bq.atom_quantize_mxfp4(x)
    _, s = check_codes(Xq, sx, x)
    assert (s == 255).sum() == 3
    back = bq.atom_dequantize_mxfp4(Xq, sx, 600, dtype=t)
    assert back.isnan().sum() == 32 + 32 + 600 - 576 and back[1, :32].isnan().all() and back[4, 576:].isnan().all()
    for many in (x[:2], x, x.repeat(40, 1)):
        Wq, sw = bq.atom_quantize_mxfp4(make(70, 600, t, 7))
        Y = bq.linear_mxfp4(many, Wq, sw)
        bad = torch.zeros(len(many), dtype=torch.bool, device="cuda")
        bad[1::6] = True
        bad[4::6] = True
        assert torch.equal(Y.isnan(), bad[:, None].expand_as(Y))


# every kind of kernel and its edges: few rows (one and two tiles), divided K, the tile sizes
SHAPES = [(1, 1, 1), (1, 17, 300), (1, 4096, 4096), (3, 130, 127), (16, 100, 11008), (17, 33, 1000), (32, 1000, 513),
          (33, 64, 128), (33, 65, 4096), (33, 65, 6145), (127, 1000, 5000), (300, 300, 300), (4000, 31, 1000), (64, 128, 2048),
          (65, 127, 4100), (100, 260, 65536), (128, 4096, 1024), (333, 777, 1155), (257, 4097, 300), (512, 8192, 256),
          (1024, 4100, 384), (4000, 4104, 200), (2304, 11008, 130), (1100, 4100, 700), (2304, 4200, 1000), (64, 4096, 8192),
          (201, 16403, 2300), (501, 16403, 2600), (1000, 10900, 4000), (777, 777, 7000), (100, 4096, 6000), (300, 777, 4100)]

# every position at which K can end in the rings of stage buffers, for each tile size (M, N, groups of K)
RINGS = ([(201, 1003, g) for g in range(1, 9)] + [(501, 501, g) for g in range(9, 14)] + [(131, 16403, g) for g in range(1, 6)] + [(131, 6003, g) for g in range(6, 14)] +
         [(201, 16403, g) for g in range(1, 5)] + [(333, 8203, 5), (333, 8203, 6)] + [(131, 11003, g) for g in range(7, 12)] +
         [(201, 16403, g) for g in range(8, 15)] + [(701, 16403, g) for g in range(5, 10)] + [(501, 16403, g) for g in range(10, 14)])


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K, dtype, bias):
    say(f"[mxfp4 linear] {M}x{N}x{K} {dtype} bias={bias}")
    t = TYPES[dtype]
    x, w = make(M, K, t, M + K), make(N, K, t, N + K + 1, 0.02)
    b = make(1, N, t, 3)[0] if bias else None
    Wq, sw = bq.atom_quantize_mxfp4(w)
    Xq, sx = bq.atom_quantize_mxfp4(x)
    Y = bq.linear_mxfp4(x, Wq, sw, bias=b)
    vx, vw = values(Xq, sx), values(Wq, sw)
    check_y(Y, vx, vw, b, K, f"{M}x{N}x{K}")
    check_y(bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, K, bias=b, dtype=t), vx, vw, b, K, f"product {M}x{N}x{K}")
    if M * N * K < 3e8:                             # the oracle's own product, from its own codes
        c, d = check_codes(Xq, sx, x), check_codes(Wq, sw, w)
        np.testing.assert_allclose((vx @ vw.t().contiguous()).cpu().numpy(), O.mx_values(*c) @ O.mx_values(*d).T, rtol=1e-9, atol=1e-9)
    need = bq.atom_gemm_mxfp4_workspace_bytes(M, N, K)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda") if need else None
    for work in (ws, None):                         # divided or not
        Y2 = bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, K, bias=b, dtype=t, workspace=work)
        check_y(Y2, vx, vw, b, K, f"{M}x{N}x{K} workspace={work is not None}")
        again = bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, K, bias=b, dtype=t, workspace=work)
        torch.testing.assert_close(again, Y2, rtol=0, atol=0)


def codes(rows, K, seed, lo=126, hi=128):
    """Random codes (every one of them) and scales, packed, with zeros behind K."""
    r = np.random.default_rng(seed)
    P = 2 * O.mx_row_bytes(K)
    c = r.integers(0, 16, (rows, P)).astype(np.uint8)
    c[:, K:] = 0
    s = r.integers(lo, hi + 1, (rows, P // 32)).astype(np.uint8)
    s[:, -(-K // 32):] = 0
    q, s3 = O.mx_pack(c, s)
    return torch.from_numpy(q).cuda(), torch.from_numpy(s3).cuda()


@pytest.mark.parametrize("M,N,K", SHAPES + [(m, n, 256 * g - 5) for m, n, g in RINGS])
def test_exact_sums(M, N, K):
    """Codes of every kind with scales 1/2, 1 and 2: products are multiples of 2^-4 and the sums of their magnitudes stay below
    2^20, so every step of fp32 is exact, in every kernel and division, and Y is the sum rounded once."""
    if K > 8000:
        K = 4096 + K % 4096
    say(f"[mxfp4 exact] {M}x{N}x{K}")
    Xq, sx = codes(M, K, 1)
    Wq, sw = codes(N, K, 2)
    vx, vw = values(Xq, sx), values(Wq, sw)
    assert float((vx.abs() @ vw.abs().t().contiguous()).max()) < 2**20
    y = vx @ vw.t().contiguous()
    need = bq.atom_gemm_mxfp4_workspace_bytes(M, N, K)
    for work in {need, 0}:
        ws = torch.full((work,), 0xA5, dtype=torch.uint8, device="cuda") if work else None
        for t in TYPES.values():
            Y = bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, K, dtype=t, workspace=ws)
            torch.testing.assert_close(Y, y.float().to(t), rtol=0, atol=0)


def test_scales_of_the_whole_range():
    """Scale bytes from 0 to 254 on either side: what fits fp32 comes out, exactly."""
    for M in (3, 40, 300):
        Xq, sx = codes(M, 256, 3, 0, 254)
        Wq, sw = codes(50, 256, 4)
        sw = 254 - sx[:, :1].expand(1, 50, 8).contiguous()               # products near 1 for the first row
        Xq, sx = Xq[:1].expand(M, 128).contiguous(), sx[:, :1].expand(1, M, 8).contiguous()
        Y = bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, 256, dtype=torch.bfloat16)
        y = values(Xq, torch.full_like(sx, 127)) @ values(Wq, torch.full_like(sw, 127)).t().contiguous()
        torch.testing.assert_close(Y, y.float().bfloat16(), rtol=0, atol=0)


# Layers of one launch: every number of columns and of waves, batches of tokens that end everywhere, rows of one group and of odd numbers.
ONE = [(1, 33, 16384), (2, 20, 8192), (3, 48, 5461), (4, 65, 4096), (4, 16, 4097), (1, 70, 16385), (2, 5, 1), (4, 1, 129), (3, 4096, 513),
       (1, 300, 255), (1, 33, 65536), (4, 20, 8192), (2, 20, 16384), (1, 5000, 300), (2, 8200, 1030), (7, 6001, 777), (16, 6000, 4096),
       (16, 4100, 2048), (16, 9000, 256), (9, 12300, 1200), (16, 12400, 300), (5, 16390, 2000), (8, 16400, 1500), (8, 20001, 8192), (13, 47, 5000),
       (16, 16384, 4096), (6, 11000, 10000), (15, 1, 4369), (8, 100, 31), (2, 4100, 32768), (1, 5000, 4097), (1, 12400, 3000), (1, 30000, 520), (17, 64, 256), (333, 250, 1155),
       (64, 4096, 4096), (128, 1000, 2048), (100, 1000, 300), (1000, 64, 520), (4095, 5, 70), (256, 1024, 1025), (31, 8190, 100), (333, 777, 1155),
       (250, 777, 2047), (20, 300, 8), (40, 64, 9), (3, 33, 15)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", ONE)
def test_one_launch_equals_two_steps(M, N, K, dtype):
    """Quantized and multiplied in one launch: the bits of the two steps where every sum is exact, also from rows that lie apart
    and start at odd elements.  Blocks' largest elements are in [4, 8) units, so that codes are halves up to 6 of one unit, and a
    sum's terms multiples of its quarter up to 36: of 2^16 terms every partial sum has 24 bits, in any order."""
    say(f"[mxfp4 one launch] {M}x{N}x{K} {dtype}")
    t = TYPES[dtype]
    K_all = K + 9

    def blocks(rows, n, seed, unit, lead):
        g = torch.Generator().manual_seed(seed)
        v = make(rows, n, t, seed).clamp(-3, 3)
        for first in lead:                           # of every block, wherever the rows begin
            at = v[:, first::32]
            v[:, first::32] = (4 + 3.9 * torch.rand(at.shape, generator=g)).to(t).cuda()
        return v * unit

    Wq, sw = bq.atom_quantize_mxfp4(blocks(N, K, 1, 2.0**-6, (0,)))
    wide = blocks(M, K_all, 2, 1, (0, 1, 3, 5, 8))
    if M > 1:
        wide[M - 1, 3:] = 0                          # a row of zeros
    wide[0, K // 2] = 7.75
    for first in (0, 1, 3, 8):
        x = wide[:, first:first + K]
        Y = bq.linear_mxfp4(x, Wq, sw)
        torch.testing.assert_close(Y, bq.atom_gemm_mxfp4(*bq.atom_quantize_mxfp4(x), Wq, sw, K, dtype=t), rtol=0, atol=0)
        torch.testing.assert_close(Y, bq.linear_mxfp4(x.contiguous(), Wq, sw), rtol=0, atol=0)
        ws = torch.empty(bq.atom_linear_mxfp4_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
        assert ws.numel() == 0
        torch.testing.assert_close(Y, bq.linear_mxfp4(x, Wq, sw, Y=torch.empty_like(Y), workspace=ws), rtol=0, atol=0)
    odd = torch.full((M, K_all), float("nan"), dtype=t, device="cuda")       # what lies around the rows is not read into them
    odd[:, 5:5 + K] = wide[:, 5:5 + K]
    torch.testing.assert_close(bq.linear_mxfp4(odd[:, 5:5 + K], Wq, sw), bq.linear_mxfp4(wide[:, 5:5 + K].contiguous(), Wq, sw),
                               rtol=0, atol=0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [s for s in ONE if s[1] < 10000])
def test_one_launch_of_any_values(M, N, K, dtype):
    """Values of any size, an outlier and a row of zeros, with a bias: within the bound of the steps."""
    t = TYPES[dtype]
    Wq, sw = bq.atom_quantize_mxfp4(make(N, K, t, 1, 0.02))
    x = make(M, K, t, 2)
    if M > 1:
        x[M - 1, 3:] = 0
    x[0, K // 2] = 1000
    b = make(1, N, t, 3)[0]
    xd, wd = (values(*q)[:, :K] for q in (bq.atom_quantize_mxfp4(x), (Wq, sw)))
    check_y(bq.linear_mxfp4(x, Wq, sw, bias=b), xd, wd, b, K, f"{M}x{N}x{K}")


@pytest.mark.parametrize("dtype", TYPES)
def test_every_value_against_every_scale(dtype):
    """Every finite value of the type in a block whose largest has each exponent from its own up: the code that the formula gives."""
    t = TYPES[dtype]
    v = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(t).cuda()
    v = torch.where(v.isfinite(), v, 0.0)
    v = torch.cat([v, torch.zeros(-v.numel() % 31, dtype=t, device="cuda")]).view(-1, 31)
    low, high = (-24, 15) if dtype == "fp16" else (-133, 127)
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device="cuda")
    for first in range(low, high + 1, 40):
        tops = torch.tensor([2.0**e for e in range(first, min(first + 40, high + 1))], dtype=torch.float64, device="cuda")
        x = torch.where(v.double().abs()[None] < 2 * tops[:, None, None], v[None], 0.0)          # the exponent of the top, or less
        x = torch.cat([x, tops.to(t)[:, None, None].expand(-1, v.shape[0], 1)], 2).reshape(-1, 32)
        x = torch.cat([x, torch.zeros(-x.shape[0] % 64, 32, dtype=t, device="cuda")])
        Xq, sx = bq.atom_quantize_mxfp4(x.view(-1, 2048))
        scale = sx.permute(1, 0, 2).reshape(-1)
        e = torch.clamp(torch.frexp(x.abs().amax(1).double())[1] - 1 - 2, -127, 125)
        e = torch.where((x != 0).any(1), e, -127)
        assert torch.equal(scale.int(), (e + 127).int())
        u = x.double().abs() * torch.exp2(-e.double())[:, None]
        code = torch.bucketize(u, border)                                   # borders below u: ties to the even code
        tie = (code < 7) & (u == border[code.clamp(max=6)]) & (code % 2 == 1)
        code = code + tie.long()
        sign = torch.signbit(x)
        got = Xq.view(-1, 16)
        got = torch.stack([got & 15, got >> 4], 2).view(-1, 32).long()
        assert torch.equal(got & 7, code)
        assert torch.equal((got >> 3)[code > 0].bool(), sign[code > 0])


def test_two_graphs_and_eager_calls_between():
    """Two captured graphs of the same shapes and eager calls in turn: none reads another's workspace."""
    for M, N, K in ((2, 300, 1000), (64, 128, 4096), (64, 4096, 8192)):      # the last divides K
        Wq, sw = bq.atom_quantize_mxfp4(make(N, K, torch.float16, 1, 0.02))
        xs = [make(M, K, torch.float16, 2 + i) for i in range(2)]
        bq.linear_mxfp4(xs[0], Wq, sw)
        torch.cuda.synchronize()
        graphs, ys = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
        for g, x in zip(graphs, xs):
            with torch.cuda.graph(g):
                ys.append(bq.linear_mxfp4(x, Wq, sw))
        for i in range(4):
            for j, x in enumerate(xs):
                x.copy_(make(M, K, torch.float16, 20 + 2 * i + j))
            streams = torch.cuda.Stream(), torch.cuda.Stream()
            for g, s in zip(graphs, streams):
                s.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(s):
                    g.replay()
            eager = [bq.linear_mxfp4(x, Wq, sw) for x in xs]
            torch.cuda.synchronize()
            for y, e in zip(ys, eager):
                torch.testing.assert_close(y, e, rtol=0, atol=0)


def test_given_buffers_and_streams():
    x, w = make(40, 700, torch.float16, 1), make(90, 700, torch.float16, 2)
    Wq, sw = bq.atom_quantize_mxfp4(w)
    want = bq.linear_mxfp4(x, Wq, sw)
    Y = torch.full((42, 90), 7.0, dtype=torch.float16, device="cuda")
    ws = torch.empty(bq.atom_linear_mxfp4_workspace_bytes(40, 90, 700), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert bq.linear_mxfp4(x, Wq, sw, Y=Y[:40], workspace=ws, stream=side) is not None
    side.synchronize()
    torch.testing.assert_close(Y[:40], want, rtol=0, atol=0)
    assert torch.all(Y[40:] == 7)                   # rows behind the last are left as they were
    with torch.cuda.stream(side):
        again = bq.linear_mxfp4(x, Wq, sw)
    other = bq.linear_mxfp4(x, Wq, sw, stream=side)
    side.synchronize()
    torch.testing.assert_close(again, want, rtol=0, atol=0)
    torch.testing.assert_close(other, want, rtol=0, atol=0)


def test_output_past_32_bits():
    """More than 2^32 bytes of Y: the last rows against a small product of their own (exact sums: any kernel's bits)."""
    M, N, K = 140000, 16384, 64
    say(f"[mxfp4 large] {M}x{N}x{K}")
    Xq, sx = codes(M, K, 5)
    Wq, sw = codes(N, K, 6)
    Y = bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, K)
    for rows in (slice(0, 40), slice(70000, 70040), slice(M - 40, M)):
        part = bq.atom_gemm_mxfp4(Xq[rows].contiguous(), sx[:, rows].contiguous(), Wq, sw, K)
        torch.testing.assert_close(Y[rows], part, rtol=0, atol=0)


def test_rows_past_32_bits():
    """More than 2^32 bytes of X: the last rows as by themselves, and back."""
    rows, K = 300000, 8192
    say(f"[mxfp4 quantize] {rows}x{K}")
    x = torch.zeros(rows, K, dtype=torch.float16, device="cuda")
    at = torch.tensor([0, 131071, 262143, 262144, rows - 1], device="cuda")
    x[at] = make(len(at), K, torch.float16, 7)
    Xq, sx = bq.atom_quantize_mxfp4(x)
    check_codes(Xq[at], sx[:, at], x[at])
    assert int((Xq != 0).any(1).sum()) == len(at)
    back = bq.atom_dequantize_mxfp4(Xq, sx, K)
    torch.testing.assert_close(back[at], bq.atom_dequantize_mxfp4(Xq[at], sx[:, at].contiguous(), K), rtol=0, atol=0)
    assert int((back != 0).any(1).sum()) == len(at)


@pytest.mark.parametrize("M,N,K", [(2100001, 3, 5), (5, 2000003, 40), (70001, 33, 300), (3, 70001, 257), (1, 200003, 1)])
def test_tall_and_wide(M, N, K):
    """Far more rows or columns than a launch has workgroups in one direction: the ends and the middle against fp64."""
    say(f"[mxfp4 linear] {M}x{N}x{K}")
    Xq, sx = codes(M, K, 7)
    Wq, sw = codes(N, K, 8)
    Y = bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, K, dtype=torch.bfloat16)
    part = lambda n: torch.cat([torch.arange(min(n, 50)), torch.arange(max(0, n // 2 - 30), n // 2), torch.arange(max(0, n - 50), n)]).cuda()  # noqa: E731
    m, n = part(M), part(N)
    y = values(Xq[m], sx[:, m]) @ values(Wq[n], sw[:, n]).t().contiguous()
    torch.testing.assert_close(Y[m][:, n], y.float().bfloat16(), rtol=0, atol=0)
    torch.testing.assert_close(Y[m], bq.atom_gemm_mxfp4(Xq[m], sx[:, m].contiguous(), Wq, sw, K, dtype=torch.bfloat16), rtol=0, atol=0)


def test_too_little_workspace():
    """Less scratch than a division needs: the undivided product's bits, and nothing written into it."""
    M, N, K = 64, 4096, 8192
    Xq, sx = bq.atom_quantize_mxfp4(make(M, K, torch.float16, 1))
    Wq, sw = bq.atom_quantize_mxfp4(make(N, K, torch.float16, 2, 0.02))
    need = bq.atom_gemm_mxfp4_workspace_bytes(M, N, K)
    assert need > 0
    want = bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, K)
    for size in (16, need - 16):
        ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
        torch.testing.assert_close(bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, K, workspace=ws), want, rtol=0, atol=0)
        assert torch.all(ws == 0xA5)
    guard = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, K, workspace=guard[:need])
    assert torch.all(guard[need:] == 0xA5)
    lin = bq.atom_linear_mxfp4_workspace_bytes(M, N, K)
    guard = torch.full((lin + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    x = make(M, K, torch.float16, 1)
    torch.testing.assert_close(bq.linear_mxfp4(x, Wq, sw, workspace=guard[:lin]), bq.linear_mxfp4(x, Wq, sw), rtol=0, atol=0)
    assert torch.all(guard[lin:] == 0xA5)


def test_outputs_stay_inside():
    """Bytes around every output of every kernel keep their values (rows and columns that end inside a tile)."""
    for M, N, K in ((3, 130, 127), (33, 65, 1000), (333, 777, 1155), (131, 6003, 300), (131, 11003, 2000), (201, 16403, 2300), (501, 16403, 2600),
                    (300, 777, 4100)):
        Xq, sx = codes(M, K, 9)
        Wq, sw = codes(N, K, 10)
        flat = torch.full((M * N + 64,), 7.0, dtype=torch.float16, device="cuda")
        Y = flat[32:32 + M * N].view(M, N)
        need = bq.atom_gemm_mxfp4_workspace_bytes(M, N, K)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
        bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, K, Y=Y, workspace=ws)
        torch.testing.assert_close(Y, bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, K, workspace=ws), rtol=0, atol=0)
        assert torch.all(flat[:32] == 7) and torch.all(flat[32 + M * N:] == 7)
