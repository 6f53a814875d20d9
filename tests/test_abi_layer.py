"""Host-side checks of the ABIs of the MXFP4 layer, the norm and the KV cache's bookkeeping (no GPU needed, no kernel is ever
launched): every declared symbol is exported, and invalid arguments are refused before any HIP call.  The addresses are
fake and never dereferenced; every call below fails validation."""
import os
import re

import pytest

import bit_quantized_gemm_amd as bq
from bit_quantized_gemm_amd import kv4_pages, mxfp4, norm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, E_NULL, E_SHAPE, E_ALIGN, E_OVERLAP = 0, 1, 2, 3, 4
A, B, C, D, E, F, G, H, I = (i << 36 for i in range(1, 10))   # aligned, far apart
S = None


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bq.lib_path()):
        pytest.skip("libatom.so not built (python -m bit_quantized_gemm_amd.build)")
    return bq.load_library()


@pytest.mark.parametrize("header,module", [("atom_mxfp4.h", mxfp4), ("atom_norm.h", norm), ("atom_kv4_pages.h", kv4_pages)])
def test_exports_every_declared_symbol(lib, header, module):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(atom_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(module.EXPORTS)
    for n in names:
        assert hasattr(lib, n), n
    for n in module.__all__:
        assert n in bq.__all__ and hasattr(bq, n), n


def test_headers_are_c(tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc")
    if not cc:
        pytest.skip("no gcc")
    src = tmp_path / "t.c"
    src.write_text('#include "atom_norm.h"\n#include "atom_kv4_pages.h"\nint main(void) { return ATOM_MX_GROUP / ATOM_MX_BLOCK; }\n')
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I" + os.path.join(ROOT, "include"), "-fsyntax-only", str(src)],
                   check=True)


def caller(fn, ok):
    return lambda **k: fn(*{**ok, **k}.values())


def test_mxfp4_sizes(lib):
    assert [bq.atom_mxfp4_row_bytes(k) for k in (1, 255, 256, 257, 4096, bq.MAX_K)] == [128, 128, 128, 256, 2048, 32768]
    assert [bq.atom_mxfp4_groups(k) for k in (1, 256, 257, bq.MAX_K)] == [1, 1, 2, 256]
    for bad in (0, -1, bq.MAX_K + 1):
        assert bq.atom_mxfp4_row_bytes(bad) == bq.atom_mxfp4_groups(bad) == -E_SHAPE


def test_quantize_and_back_validation(lib):
    q = caller(lib.atom_quantize_mxfp4, dict(x=A, ldx=100, t=0, rows=4, k=100, xq=B, sx=C, s=S))
    for n in ("x", "xq", "sx"):
        assert q(**{n: None}) == E_NULL
    for bad in (dict(rows=0), dict(rows=(1 << 24) + 1), dict(k=0), dict(k=65537, ldx=70000), dict(t=2), dict(t=-1), dict(ldx=99)):
        assert q(**bad) == E_SHAPE, bad
    assert q(x=A + 1) == q(xq=B + 8) == q(sx=C + 4) == E_ALIGN
    assert q(ldx=1000, xq=A + 6016) == q(sx=B + 496) == q(xq=A + 16) == E_OVERLAP      # X spans 2 * 3100 bytes, the codes 4 * 128
    d = caller(lib.atom_dequantize_mxfp4, dict(xq=A, sx=B, rows=4, k=100, t=0, x=C, s=S))
    for n in ("x", "xq", "sx"):
        assert d(**{n: None}) == E_NULL
    assert d(rows=0) == d(k=0) == d(t=2) == E_SHAPE
    assert d(xq=A + 8) == d(sx=B + 8) == d(x=C + 2) == E_ALIGN
    assert d(x=A + 496) == d(x=B + 16) == E_OVERLAP
    w = caller(lib.atom_dequantize_w8a8, dict(xq=A, sx=B, rows=4, k=100, t=0, x=C, s=S))
    for n in ("x", "xq", "sx"):
        assert w(**{n: None}) == E_NULL
    assert w(rows=0) == w(k=0) == w(t=2) == E_SHAPE
    assert w(xq=A + 8) == w(sx=B + 8) == w(x=C + 2) == E_ALIGN
    assert w(x=A + 496) == w(x=B) == E_OVERLAP


def test_gemm_and_linear_validation(lib):
    g = caller(lib.atom_gemm_mxfp4, dict(xq=A, sx=B, wq=C, sw=D, bias=None, m=4, n=4, k=300, t=0, y=E, ws=None, nws=0, s=S))
    for n in ("xq", "sx", "wq", "sw", "y"):
        assert g(**{n: None}) == E_NULL
    assert g(m=0) == g(n=0) == g(k=0) == g(t=5) == g(k=65537) == g(m=1 << 24, n=1 << 24) == E_SHAPE
    for n, p in (("xq", A), ("sx", B), ("wq", C), ("sw", D), ("y", E), ("bias", F)):
        assert g(**{n: p + 4}) == E_ALIGN
    assert g(y=A + 16) == g(y=C + 1008) == g(y=D + 48) == g(bias=F, y=F) == E_OVERLAP
    need = bq.atom_gemm_mxfp4_workspace_bytes(64, 4096, 11008)
    assert need > 0
    assert g(m=64, n=4096, k=11008, ws=F + 4, nws=need) == E_ALIGN
    assert g(m=64, n=4096, k=11008, ws=E, nws=need) == E_OVERLAP
    assert lib.atom_gemm_mxfp4_workspace_bytes(0, 4, 4) == lib.atom_linear_mxfp4_workspace_bytes(4, 0, 4) == -E_SHAPE
    assert bq.atom_linear_mxfp4_workspace_bytes(4, 4, 256) == 0          # one launch: nothing to keep
    assert bq.atom_linear_mxfp4_workspace_bytes(16, 4, 4096) == 0 < bq.atom_linear_mxfp4_workspace_bytes(16, 4, 4097)
    need = bq.atom_linear_mxfp4_workspace_bytes(17, 4, 4352)
    assert need >= 17 * (2176 + 136)
    f = caller(lib.atom_linear_mxfp4, dict(x=A, ldx=4352, t=0, wq=C, sw=D, bias=None, m=17, n=4, k=4352, y=E, ws=F, nws=need, s=S))
    for n in ("x", "wq", "sw", "y", "ws"):
        assert f(**{n: None}) == E_NULL
    assert f(nws=need - 1) == f(ldx=4351) == f(t=-1) == f(k=0) == E_SHAPE
    assert f(x=A + 1) == f(ws=F + 8) == f(y=E + 2) == f(sw=D + 8) == E_ALIGN
    assert f(y=F) == f(ws=A) == f(y=C) == f(y=D) == E_OVERLAP


@pytest.mark.parametrize("name", norm.EXPORTS)
def test_norm_validation(lib, name):
    f = caller(getattr(lib, name), dict(x=A, ldx=100, r=B, ldr=100, w=C, eps=1e-6, t=0, rows=4, k=100, h=D, ldh=100, xq=E, sx=F, s=S))
    for n in ("x", "w", "xq", "sx", "h"):
        assert f(**{n: None}) == E_NULL
    for bad in (dict(rows=0), dict(k=0), dict(k=65537), dict(t=2), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(ldx=99), dict(ldr=99), dict(ldh=99), dict(r=None)):
        assert f(**bad) == E_SHAPE, bad
    for n, p in (("x", A), ("r", B), ("w", C), ("h", D)):
        assert f(**{n: p + 1}) == E_ALIGN
    assert f(xq=E + 8) == f(sx=F + 4) == E_ALIGN
    for bad in (dict(xq=A + 16), dict(xq=B + 16), dict(xq=C + 16), dict(sx=A), dict(sx=E + 16), dict(xq=D + 16), dict(sx=D),
                dict(h=C), dict(h=A + 2), dict(h=B + 2), dict(h=A, ldh=101), dict(h=B, ldh=104), dict(h=E)):
        assert f(**bad) == E_OVERLAP, bad
    assert f(r=A + 64, h=A + 64) == E_OVERLAP                            # in place of one term, over the other


def test_pages_validation(lib):
    e = caller(lib.atom_kv4_extend, dict(lens=A, new=B, table=C, batch=4, width=8, page=16, free=D, cap=100, state=E, slots=F, total=20,
                                         start=G, out=H, sout=I, s=S))
    for n in ("lens", "new", "table", "free", "state", "slots", "start", "out", "sout"):
        assert e(**{n: None}) == E_NULL
    for bad in (dict(batch=0), dict(batch=(1 << 20) + 1), dict(width=0), dict(page=8), dict(page=24), dict(page=512), dict(page=-16),
                dict(width=1 << 27), dict(cap=0), dict(cap=(1 << 27) + 1), dict(total=0), dict(total=(1 << 24) + 1)):
        assert e(**bad) == E_SHAPE, bad
    for n, p in (("lens", A), ("new", B), ("table", C), ("free", D), ("state", E), ("start", G), ("out", H), ("sout", I)):
        assert e(**{n: p + 2}) == E_ALIGN
    assert e(slots=F + 4) == E_ALIGN
    for bad in (dict(slots=B), dict(table=D), dict(start=A), dict(out=A + 4), dict(out=B), dict(sout=E + 4), dict(sout=A), dict(start=F),
                dict(out=E), dict(table=A), dict(lens=C, out=C), dict(lens=C + 4, out=C + 4), dict(sout=H)):
        assert e(**bad) == E_OVERLAP, bad
    r = caller(lib.atom_kv4_release, dict(done=A, lens=B, table=C, batch=4, width=8, page=16, free=D, cap=100, state=E, out=F, sout=G, s=S))
    for n in ("done", "lens", "table", "free", "state", "out", "sout"):
        assert r(**{n: None}) == E_NULL
    for bad in (dict(batch=0), dict(width=0), dict(page=17), dict(cap=0), dict(width=1 << 27)):
        assert r(**bad) == E_SHAPE, bad
    for n, p in (("lens", B), ("table", C), ("free", D), ("state", E), ("out", F), ("sout", G)):
        assert r(**{n: p + 2}) == E_ALIGN
    for bad in (dict(free=C), dict(out=A), dict(out=B + 4), dict(sout=E + 4), dict(out=D + 396), dict(sout=F), dict(free=B)):
        assert r(**bad) == E_OVERLAP, bad


class _NoLaunch:
    """The loaded library with every entry point that would enqueue work replaced by a failure."""

    def __init__(self, lib):
        self._lib = lib

    def __getattr__(self, name):
        if name.endswith(("_bytes", "_groups", "strerror")):
            return getattr(self._lib, name)

        def fail(*a):
            raise AssertionError(f"{name} was called with arguments the binding should have refused")
        return fail


def test_binding_refusals(lib, monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(bq, "_LIB", _NoLaunch(lib))
    z, f16, b16, f32, i8, u8, i32, i64 = (torch.zeros, torch.float16, torch.bfloat16, torch.float32, torch.int8,
                                          torch.uint8, torch.int32, torch.int64)
    X, W = z((4, 300), dtype=f16), z((300,), dtype=f16)
    Xq, sx, Wq, sw = z((4, 256), dtype=u8), z((2, 4, 8), dtype=u8), z((6, 256), dtype=u8), z((2, 6, 8), dtype=u8)
    Q8, s8 = z((4, 384), dtype=i8), z((4,), dtype=f32)
    lens, new, table, pool = z(5, dtype=i32), z(5, dtype=i32), z((5, 3), dtype=i32), bq.kv4_pool(9, device="cpu")
    done = z(5, dtype=torch.bool)
    shape = [
        lambda: bq.atom_quantize_mxfp4(X[0]),
        lambda: bq.atom_quantize_mxfp4(X, Xq=z((4, 300), dtype=u8)),
        lambda: bq.atom_quantize_mxfp4(X, sx=z((4, 2, 8), dtype=u8)),
        lambda: bq.atom_dequantize_mxfp4(Xq, sx, 600),
        lambda: bq.atom_dequantize_mxfp4(Xq, z((2, 5, 8), dtype=u8), 300),
        lambda: bq.atom_dequantize_mxfp4(Xq, sx, 300, X=z((4, 301), dtype=f16)),
        lambda: bq.atom_dequantize_w8a8(Q8, s8, 400),
        lambda: bq.atom_dequantize_w8a8(Q8, s8[:3], 300),
        lambda: bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, 600),
        lambda: bq.atom_gemm_mxfp4(Xq, sx, Wq, sw[:1], 300),
        lambda: bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, 300, bias=z((4,), dtype=f16)),
        lambda: bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, 300, Y=z((6, 4), dtype=f16)),
        lambda: bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, 300, workspace=z((8, 8), dtype=u8)),
        lambda: bq.linear_mxfp4(X, z((6, 150), dtype=u8), sw),
        lambda: bq.linear_mxfp4(X, Wq, sw[:, :5]),
        lambda: bq.linear_mxfp4(z((9, 8000), dtype=f16), z((6, 4096), dtype=u8), z((32, 6, 8), dtype=u8), workspace=z((16,), dtype=u8)),
        lambda: bq.atom_rmsnorm_w8a8(X, W[:299]),
        lambda: bq.atom_rmsnorm_w8a8(X, W, residual=X[:3]),
        lambda: bq.atom_rmsnorm_w8a8(X, W, residual=X, H=X[:, :200]),
        lambda: bq.atom_rmsnorm_mxfp4(X, W, Xq=z((4, 150), dtype=u8)),
        lambda: bq.atom_rmsnorm_mxfp4(X[0], W),
        lambda: bq.atom_kv4_extend(lens[:4], new, table, pool, 16, 7),
        lambda: bq.atom_kv4_extend(lens, new[:4], table, pool, 16, 7),
        lambda: bq.atom_kv4_extend(lens, new, table[0], pool, 16, 7),
        lambda: bq.atom_kv4_extend(lens, new, table, pool._replace(free=table), 16, 7),
        lambda: bq.atom_kv4_extend(lens, new, table, pool._replace(state=lens), 16, 7),
        lambda: bq.atom_kv4_extend(lens, new, table, pool, 16, 7, slots=z(8, dtype=i64)),
        lambda: bq.atom_kv4_extend(lens, new, table, pool, 16, 7, q_start=z(5, dtype=i32)),
        lambda: bq.atom_kv4_release(done[:4], lens, table, pool, 16),
        lambda: bq.atom_kv4_release(done, lens, table, pool, 16, state_out=lens),
    ]
    for i, call in enumerate(shape):
        with pytest.raises(bq.AtomError, match="shape|-D"):
            print(i)
            call()
    kind = [
        lambda: bq.atom_quantize_mxfp4(X.float()),
        lambda: bq.atom_dequantize_mxfp4(Xq, sx, 300, dtype=f32),
        lambda: bq.atom_dequantize_mxfp4(Xq.view(i8), sx, 300),
        lambda: bq.atom_dequantize_w8a8(Q8.view(u8), s8, 300),
        lambda: bq.linear_mxfp4(X, Wq, sw, bias=z((6,), dtype=b16)),
        lambda: bq.linear_mxfp4(X, Wq.view(i8), sw),
        lambda: bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, 300, dtype=f32),
        lambda: bq.atom_rmsnorm_w8a8(X, W.bfloat16()),
        lambda: bq.atom_rmsnorm_w8a8(X, W, residual=X.bfloat16()),
        lambda: bq.atom_rmsnorm_mxfp4(X, W, residual=X, H=X.bfloat16()),
        lambda: bq.atom_rmsnorm_mxfp4(X, W, H=X),
        lambda: bq.atom_rmsnorm_mxfp4(X, W, Xq=Q8[:, :256].contiguous()),
        lambda: bq.atom_kv4_extend(lens.long(), new, table, pool, 16, 7),
        lambda: bq.atom_kv4_extend(lens, new, table, pool, 16, 0),
        lambda: bq.atom_kv4_extend(lens, new, table, pool, 16, 7, slots=z(7, dtype=i32)),
        lambda: bq.atom_kv4_extend(lens, new, table.t().contiguous().t(), pool, 16, 7),
        lambda: bq.atom_kv4_release(done.to(u8), lens, table, pool, 16),
        lambda: bq.atom_kv4_release(done, lens, table, None, 16),
    ]
    for i, call in enumerate(kind):
        with pytest.raises(bq.AtomError, match="must be"):
            print(i)
            call()
    with pytest.raises(bq.AtomError, match="agree"):
        bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, 300, bias=z((6,), dtype=b16), dtype=f16)
    cols = z((300, 4), dtype=f16).t()
    for call in (lambda: bq.linear_mxfp4(cols, Wq, sw), lambda: bq.linear_mxfp4(X[:1].expand(4, 300), Wq, sw),
                 lambda: bq.atom_rmsnorm_w8a8(cols, W), lambda: bq.atom_rmsnorm_w8a8(X, W, residual=X[:1].expand(4, 300))):
        with pytest.raises(bq.AtomError, match="contiguous|ROCm device"):
            call()
    # well-formed host tensors get as far as the device check
    for i, call in enumerate((lambda: bq.atom_quantize_mxfp4(X), lambda: bq.linear_mxfp4(X, Wq, sw), lambda: bq.atom_dequantize_mxfp4(Xq, sx, 300),
                              lambda: bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, 300), lambda: bq.atom_rmsnorm_w8a8(X, W),
                              lambda: bq.atom_rmsnorm_mxfp4(X, W, residual=X), lambda: bq.atom_dequantize_w8a8(Q8, s8, 300),
                              lambda: bq.atom_kv4_extend(lens, new, table, pool, 16, 7), lambda: bq.atom_kv4_release(done, lens, table, pool, 16))):
        with pytest.raises(bq.AtomError, match="ROCm device"):
            print(i)
            call()


def test_short_calls_leave_the_rest_to_the_full_checks(lib):
    """The extension module takes plain device tensors alone: anything else is None, whatever it is, and no Python error."""
    torch = pytest.importorskip("torch")
    short = bq._SHORT
    if short is None:
        pytest.skip("_short.so not built (python -m bit_quantized_gemm_amd.build)")
    t, i = torch.zeros((4, 300), dtype=torch.float16), torch.zeros(5, dtype=torch.int32)

    class Sub(torch.Tensor):
        pass
    odd = [None, 0, 1.5, "x", [t], t, i, t.numpy(), t.as_subclass(Sub), torch.nn.Parameter(t), object(), 1 << 80, -1]
    sizes = {"quantize_mxfp4": 1, "linear_mxfp4": 4, "gemm_mxfp4": 8, "dequantize_mxfp4": 4, "dequantize_w8a8": 4, "rmsnorm_w8a8": 4, "rmsnorm_mxfp4": 4,
             "kv4_extend": 7, "kv4_release": 6}
    for name, n in sizes.items():
        f = getattr(short, name)
        for k in range(n + 2):                       # wrong numbers of arguments too
            for o in odd:
                assert f(*[o] * k) is None, (name, k, o)
        for a in odd:
            for b in odd:
                assert f(*([a, b] * n)[:n]) is None, (name, a, b)
    for bad in ((), ({},), ([], None), ({"atom_kv4_extend": "x"}, None)):
        with pytest.raises(TypeError):
            short.bind(*bad)
    assert bq._bind_short(lib, ("atom_linear_mxfp4",)) is short           # (names left out: those calls return None)
    assert short.quantize_mxfp4(t) is None
    assert bq._bind_short(lib, [n for m in (mxfp4, norm, kv4_pages) for n in m.EXPORTS] + ["atom_dequantize_w8a8"]) is short
