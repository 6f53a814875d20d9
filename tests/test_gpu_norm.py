"""The norm in front of the quantized layers on the GPU against the CPU oracle (needs an MI355X): sums, codes and scales bit for
bit; the oracle's norm is in fp64, where two formulas for one value differ by a few 2^-53 of it, far from the next border for
any of these inputs (a border within 2^-50 of one of 10^7 values has a chance of 10^-7)."""
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


def make(rows, K, t, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g) * gain
    x[:, torch.randint(0, K, (max(1, K // 100),), generator=g)] *= 20
    return x.to(t).cuda()


def weights(K, t, seed=9):
    return (torch.randn(K, generator=torch.Generator().manual_seed(seed)) * 0.3 + 1).to(t).cuda()


def check(x, w, eps, r=None, given=None, **k):
    """Both norms of x (+ r) against the oracle; `given`: what the calls read, where that is not x, w and r themselves."""
    t = x.dtype
    y, h = O.rmsnorm(f32(x), f32(w), eps, None if r is None else f32(r),
                     lambda v: torch.from_numpy(v).to(t).float().numpy())
    a = (x, w, r) if given is None else given
    for call in (bq.atom_rmsnorm_w8a8, bq.atom_rmsnorm_mxfp4):
        Xq, sx, H = call(a[0], a[1], eps, residual=a[2], **k)
        if r is None:
            assert H is None
        else:
            np.testing.assert_array_equal(f32(H), h)
        if call is bq.atom_rmsnorm_w8a8:
            q, s = O.w8_codes(y)
            np.testing.assert_array_equal(sx.cpu().numpy().view(np.uint32), s.view(np.uint32))
        else:
            q, s = O.mx_pack(*O.mx_codes(y))
            np.testing.assert_array_equal(sx.cpu().numpy(), s)
        np.testing.assert_array_equal(Xq.cpu().numpy(), q)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 7), (5, 33), (4, 256), (9, 257), (2, 512), (7, 520), (6, 2048), (5, 2049), (3, 4096),
                                    (3, 4097), (2, 8192), (2, 11008), (3, 16384), (2, 16385), (2, 65536), (1, 65535), (385, 520),
                                    (390, 1155), (400, 2048), (1025, 8192), (1026, 5001)])
def test_norm(rows, K, dtype, residual):
    say(f"[norm] {rows}x{K} {dtype} residual={residual}")
    t = TYPES[dtype]
    check(make(rows, K, t, rows + K), weights(K, t), 1e-5, make(rows, K, t, rows + K + 1, 3.0) if residual else None)


@pytest.mark.parametrize("dtype", TYPES)
def test_many_rows(dtype):
    """Enough values for the borders that 32 bits cannot decide: about one in 2^16 (int8) and 2^18 (MXFP4) of 2^24."""
    t = TYPES[dtype]
    say(f"[norm] 4096x4096 {dtype}")
    check(make(4096, 4096, t, 1), weights(4096, t), 1e-6, make(4096, 4096, t, 2))


@pytest.mark.parametrize("dtype", TYPES)
def test_magnitudes(dtype):
    """Rows of zeros and of one value, of one large value, rows over the type's range, weights of zero and of either sign."""
    t = TYPES[dtype]
    x = make(12, 700, t, 3).float()
    x[0] = 0
    x[1] = 0
    x[1, 5] = 3.0
    x[2] = 1.0
    x[3] *= 2.0**-14
    x[4] *= 2.0**-24
    x[5] *= 300
    x[6] = -x[6].abs()
    if dtype == "bf16":
        x[7] *= 2.0**-90
        x[8] *= 2.0**60
        x[9] *= 2.0**100
    x = x.to(t)
    w = weights(700, t).clone()
    w[::7] = 0
    w[3::5] *= -1
    for eps in (1e-6, 1e-12, 1.0, 1e-30):
        check(x, w, eps)
        check(x, w, eps, torch.zeros_like(x))
    check(x, torch.zeros_like(w), 1e-5)


@pytest.mark.parametrize("dtype", TYPES)
def test_borders(dtype):
    """Rows whose norm is a power of two or one: values that lie exactly on the borders of codes and blocks."""
    t = TYPES[dtype]
    rows = []
    for a in (1.0, 2.0, 0.25):
        r = torch.zeros(256)
        r[:4] = a * 8                                  # sum 4 a^2 64 over 256: mean a^2
        rows.append(r)
        rows.append(torch.full((256,), a) * torch.where(torch.arange(256) % 2 == 0, 1.0, -1.0))
    x = torch.stack(rows).to(t).cuda()
    border = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0, 63.5, 62.5, 127.0, 254.0])
    for s in range(4):
        w = torch.cat([border, -border]).repeat(8)[:256].roll(s).to(t).cuda()
        check(x, w, 1e-40)                             # eps below any bit of the mean


def test_rows_apart_shifted_and_in_place():
    t = torch.float16
    X, R = make(40, 1000, t, 5), make(40, 1000, t, 6)
    w = weights(1001, t)
    for cols in (slice(0, 512), slice(8, 520), slice(1, 514), slice(3, 700)):
        n = cols.stop - cols.start
        check(X[:, cols], w[:n], 1e-5, R[:, cols])
        check(X[::3, cols], w[:n], 1e-5, R[::3, cols])
    check(X[2:3, 5:], w[:995], 1e-5, R[3:4, 5:])
    off = torch.empty(1001, dtype=t, device="cuda")[1:]        # weights that no wide load fits
    off.copy_(w[:1000])
    check(X, off, 1e-5, R)
    for call in (bq.atom_rmsnorm_w8a8, bq.atom_rmsnorm_mxfp4):
        want = call(X, w[:1000], residual=R)
        for place in ("residual", "x", "slice"):
            x, r = X.clone(), R.clone()
            if place == "slice":
                wide = torch.full((40, 1100), 7.0, dtype=t, device="cuda")
                r = wide[:, 16:1016]
                r.copy_(R)
            Xq, sx, H = call(x, w[:1000], residual=r, H=x if place == "x" else r)
            assert H is (x if place == "x" else r)
            for a, b in zip((Xq, sx, H), want):
                torch.testing.assert_close(a, b, rtol=0, atol=0)
            if place == "slice":
                assert torch.all(wide[:, :16] == 7) and torch.all(wide[:, 1016:] == 7)
            else:
                torch.testing.assert_close(r if place == "x" else x, R if place == "x" else X, rtol=0, atol=0)


def test_survives_inf_and_nan():
    """No fault, and the rows beside them are right."""
    x, w = make(9, 600, torch.float16, 6), weights(600, torch.float16)
    bad = x.clone()
    bad[1, 3], bad[4, 599], bad[7] = float("inf"), float("nan"), -float("inf")
    keep = [0, 2, 3, 5, 6, 8]
    for call in (bq.atom_rmsnorm_w8a8, bq.atom_rmsnorm_mxfp4):
        (a, sa, _), (b, sb, _) = call(x, w), call(bad, w)
        torch.testing.assert_close(a[keep], b[keep], rtol=0, atol=0)
        if sa.dim() == 1:
            torch.testing.assert_close(sa[keep], sb[keep], rtol=0, atol=0)
        else:
            torch.testing.assert_close(sa[:, keep], sb[:, keep], rtol=0, atol=0)


def test_given_buffers_streams_and_graphs():
    t = torch.bfloat16
    X, R, w = make(50, 1000, t, 1), make(50, 1000, t, 2), weights(1000, t)
    for call, shapes in ((bq.atom_rmsnorm_w8a8, ((52, 1024), torch.int8, (52,), torch.float32)),
                         (bq.atom_rmsnorm_mxfp4, ((52, 512), torch.uint8, None, torch.uint8))):
        want = call(X, w, residual=R)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        Xq = torch.full(shapes[0], 77, dtype=shapes[1], device="cuda")
        sx = torch.full(shapes[2] if shapes[2] else (4, 50, 8), 77, dtype=shapes[3], device="cuda")
        H = torch.empty_like(X)
        side.wait_stream(torch.cuda.current_stream())
        got = call(X, w, residual=R, H=H, Xq=Xq[:50], sx=sx[:50] if shapes[2] else sx, stream=side)
        side.synchronize()
        for a, b in zip(got, want):
            torch.testing.assert_close(a, b, rtol=0, atol=0)
        assert torch.all(Xq[50:] == 77) and (not shapes[2] or torch.all(sx[50:] == 77))
        other = call(X, w, residual=R, stream=side)
        side.synchronize()
        for a, b in zip(other, want):
            torch.testing.assert_close(a, b, rtol=0, atol=0)
        graph = torch.cuda.CUDAGraph()
        r = R.clone()
        with torch.cuda.graph(graph):
            out = call(X, w, residual=r, H=r)          # the residual replaced: each replay adds X once more
        keep = R.clone()
        for i in range(4):
            r.copy_(keep)
            graph.replay()
            eager = call(X, w, residual=keep)
            torch.cuda.synchronize()
            for a, b in zip(out, eager):
                torch.testing.assert_close(a, b, rtol=0, atol=0)
            keep = eager[2]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 127), (5, 128), (4, 129), (7, 1155), (300, 4096)])
def test_dequantize_w8a8(rows, K, dtype):
    t = TYPES[dtype]
    Xq, sx = bq.atom_quantize_w8a8(make(rows, K, t, 1))
    want = (Xq[:, :K].float() * sx[:, None]).to(t)
    torch.testing.assert_close(bq.atom_dequantize_w8a8(Xq, sx, K, dtype=t), want, rtol=0, atol=0)
    X = torch.full((rows + 1, K), 7.0, dtype=t, device="cuda")
    assert bq.atom_dequantize_w8a8(Xq, sx, K, X=X[:rows]).dtype is t
    torch.testing.assert_close(X[:rows], want, rtol=0, atol=0)
    assert torch.all(X[rows] == 7)


def test_rows_past_32_bits():
    """More than 2^32 bytes of X, and of H: the last rows as by themselves."""
    rows, K, t = 300000, 8192, torch.bfloat16
    say(f"[norm] {rows}x{K}")
    x, w = torch.zeros(rows, K, dtype=t, device="cuda"), weights(K, t)
    at = torch.tensor([0, 131071, 262143, 262144, rows - 1], device="cuda")
    x[at] = make(len(at), K, t, 7)
    for call in (bq.atom_rmsnorm_w8a8, bq.atom_rmsnorm_mxfp4):
        Xq, sx, H = call(x, w, 1e-5, residual=x)
        q, s, h = call(x[at], w, 1e-5, residual=x[at])
        torch.testing.assert_close(Xq[at], q, rtol=0, atol=0)
        torch.testing.assert_close(sx[at] if sx.dim() == 1 else sx[:, at], s, rtol=0, atol=0)
        torch.testing.assert_close(H[at], h, rtol=0, atol=0)
        some = Xq != 0 if Xq.dtype == torch.int8 else (Xq & 0x77) != 0      # (a zero keeps its sign: a negative weight's)
        assert int(some.any(1).sum()) == int((H != 0).any(1).sum()) == len(at)


def test_scales_next_to_nothing():
    """bf16 weights so small that a row's scale is one of fp32's smallest numbers: codes stay within +-127."""
    x = make(6, 300, torch.bfloat16, 4)
    for e in (-118, -126, -130, -133):
        w = torch.full((300,), 2.0**e, device="cuda").bfloat16()
        y, _ = O.rmsnorm(f32(x), f32(w), 1e-6)
        if e > -120:
            check(x, w, 1e-6)
        Xq, sx, _ = bq.atom_rmsnorm_w8a8(x, w, 1e-6)
        assert int(Xq.min()) >= -127
        # products below 2^-126 are rounded to steps of 2^-149, which is up to 2^-149 / 2 of y / h before the factor
        back = Xq[:, :300].double().cpu().numpy() * sx.double().cpu().numpy()[:, None]
        assert (np.abs(back - y) <= np.abs(y).max(1, keepdims=True) * 2.0**-6 + 2.0**-147).all()
