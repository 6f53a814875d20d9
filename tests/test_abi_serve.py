"""Host-side checks of the W8A8 and KV cache ABIs (no GPU needed, no kernel is ever launched): every
declared symbol is exported, and invalid arguments are refused before any HIP call.  The addresses are
fake and never dereferenced; every call below fails validation."""
import ctypes
import os
import re

import pytest

import bit_quantized_gemm_amd as bq
from bit_quantized_gemm_amd import kv4, w8a8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, E_NULL, E_SHAPE, E_ALIGN, E_OVERLAP = 0, 1, 2, 3, 4
A, B, C, D, E, F, G, H = (i << 36 for i in range(1, 9))   # aligned, far apart
S = None


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bq.lib_path()):
        pytest.skip("libatom.so not built (python -m bit_quantized_gemm_amd.build)")
    return bq.load_library()


@pytest.mark.parametrize("header,exports", [("atom_w8a8.h", w8a8.EXPORTS), ("atom_kv4.h", kv4.EXPORTS)])
def test_exports_every_declared_symbol(lib, header, exports):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(atom_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(exports)
    for n in names:
        assert hasattr(lib, n), n
    for n in w8a8.__all__ + kv4.__all__:
        assert n in bq.__all__ and hasattr(bq, n), n


def test_headers_are_c(tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc")
    if not cc:
        pytest.skip("no gcc")
    src = tmp_path / "t.c"
    src.write_text('#include "atom_kv4.h"\nint main(void) { atom_kv4_cache c; (void)c; return ATOM_BF16 - 1; }\n')
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I" + os.path.join(ROOT, "include"), "-fsyntax-only", str(src)],
                   check=True)


def test_w8a8_row_bytes(lib):
    assert [bq.atom_w8a8_row_bytes(k) for k in (1, 127, 128, 129, 4096, bq.MAX_K)] == [128, 128, 128, 256, 4096, 65536]
    for bad in (0, -1, bq.MAX_K + 1):
        assert bq.atom_w8a8_row_bytes(bad) == -E_SHAPE


def test_quantize_w8a8_validation(lib):
    q = lib.atom_quantize_w8a8
    assert q(None, 100, 0, 4, 100, B, C, S) == E_NULL
    assert q(A, 100, 0, 4, 100, None, C, S) == E_NULL
    assert q(A, 100, 0, 4, 100, B, None, S) == E_NULL
    assert q(A, 100, 0, 0, 100, B, C, S) == E_SHAPE
    assert q(A, 100, 0, 4, 0, B, C, S) == E_SHAPE
    assert q(A, 70000, 0, 4, 65537, B, C, S) == E_SHAPE
    assert q(A, 100, 2, 4, 100, B, C, S) == E_SHAPE           # no such type
    assert q(A, 99, 0, 4, 100, B, C, S) == E_SHAPE            # rows would overlap
    assert q(A + 1, 100, 0, 4, 100, B, C, S) == E_ALIGN
    assert q(A, 100, 0, 4, 100, B + 8, C, S) == E_ALIGN
    assert q(A, 100, 0, 4, 100, B, C + 4, S) == E_ALIGN
    assert q(A, 1000, 0, 4, 100, A + 6016, C, S) == E_OVERLAP  # X spans 2 * 3100 bytes
    assert q(A, 100, 0, 4, 100, B, B + 256, S) == E_OVERLAP    # scales inside the codes (4 x 128 bytes)


def test_gemm_w8a8_validation(lib):
    g = lib.atom_gemm_w8a8
    ok = (A, B, C, D, None, 4, 4, 256, 0, E, None, 0, S)

    def call(**k):
        names = ("xq", "sx", "wq", "sw", "bias", "m", "n", "k", "t", "y", "ws", "nws", "s")
        return g(*[k.get(n, v) for n, v in zip(names, ok)])
    for n in ("xq", "sx", "wq", "sw", "y"):
        assert call(**{n: None}) == E_NULL
    assert call(m=0) == call(n=0) == call(k=0) == call(t=5) == call(k=65537) == E_SHAPE
    assert call(m=1 << 24, n=1 << 24) == E_SHAPE
    for n, p in (("xq", A), ("sx", B), ("wq", C), ("sw", D), ("y", E), ("bias", F)):
        assert call(**{n: p + 4}) == E_ALIGN
    assert call(y=A + 16) == call(y=C + 512) == E_OVERLAP
    assert call(bias=F, y=F) == E_OVERLAP
    need = bq.atom_gemm_w8a8_workspace_bytes(64, 128, 8192)
    assert need > 0
    assert call(m=64, n=128, k=8192, ws=F + 4, nws=need) == E_ALIGN
    assert call(m=64, n=128, k=8192, ws=E, nws=need) == E_OVERLAP
    assert lib.atom_gemm_w8a8_workspace_bytes(0, 4, 4) == -E_SHAPE


def test_linear_w8a8_validation(lib):
    g = lib.atom_linear_w8a8
    assert bq.atom_linear_w8a8_workspace_bytes(4, 4, 256) == 0               # one launch: nothing to keep
    need = bq.atom_linear_w8a8_workspace_bytes(8, 4, 256)
    assert need >= 8 * 256 + 32
    ok = (A, 256, 0, C, D, None, 8, 4, 256, E, F, need, S)

    def call(**k):
        names = ("x", "ldx", "t", "wq", "sw", "bias", "m", "n", "k", "y", "ws", "nws", "s")
        return g(*[k.get(n, v) for n, v in zip(names, ok)])
    for n in ("x", "wq", "sw", "y", "ws"):
        assert call(**{n: None}) == E_NULL
    assert call(nws=need - 1) == call(ldx=255) == call(t=-1) == call(k=0) == E_SHAPE
    assert call(x=A + 1) == call(ws=F + 8) == call(y=E + 2) == E_ALIGN
    assert call(y=F) == call(ws=A) == call(y=C) == E_OVERLAP


def _c(k=A, kp=B, v=C, vp=D, pages=4, page=16, heads=2, dim=64):
    return kv4._CCache(k, kp, v, vp, pages, page, heads, dim)


def test_append_and_read_validation(lib):
    a, r = lib.atom_kv4_append, lib.atom_kv4_read
    assert a(None, 128, F, 128, G, 3, 0, _c(), S) == E_NULL
    assert a(E, 128, None, 128, G, 3, 0, _c(), S) == E_NULL
    assert a(E, 128, F, 128, None, 3, 0, _c(), S) == E_NULL
    assert a(E, 128, F, 128, G, 3, 0, _c(k=None), S) == E_NULL
    assert a(E, 128, F, 128, G, 3, 0, None, S) == E_NULL
    for bad in (dict(dim=96), dict(page=24), dict(page=8), dict(page=512), dict(pages=0), dict(heads=0),
                dict(heads=1025), dict(pages=1 << 27)):
        assert a(E, 1 << 20, F, 1 << 20, G, 3, 0, _c(**bad), S) == E_SHAPE, bad
    assert a(E, 128, F, 128, G, 0, 0, _c(), S) == E_SHAPE
    assert a(E, 128, F, 128, G, 3, 3, _c(), S) == E_SHAPE
    assert a(E, 120, F, 128, G, 3, 0, _c(), S) == E_SHAPE
    assert a(E, 132, F, 128, G, 3, 0, _c(), S) == E_ALIGN
    assert a(E + 8, 128, F, 128, G, 3, 0, _c(), S) == E_ALIGN
    assert a(E, 128, F, 128, G + 4, 3, 0, _c(), S) == E_ALIGN
    assert a(E, 128, F, 128, G, 3, 0, _c(vp=D + 4), S) == E_ALIGN
    assert a(E, 128, A + 1024, 128, G, 3, 0, _c(), S) == E_OVERLAP          # V inside k
    assert a(E, 128, F, 128, G, 3, 0, _c(v=A + 1024), S) == E_OVERLAP       # k over v
    assert r(_c(), G, 3, 0, None, F, S) == E_NULL
    assert r(_c(), None, 3, 0, E, F, S) == E_NULL
    assert r(_c(dim=65), G, 3, 0, E, F, S) == E_SHAPE
    assert r(_c(), G, 3, 2, E, F, S) == E_SHAPE
    assert r(_c(), G, 3, 0, E + 2, F, S) == E_ALIGN
    assert r(_c(), G, 3, 0, E, E + 512, S) == E_OVERLAP                     # 3 x 2 x 64 x 2 = 768 bytes
    assert r(_c(), G, 3, 0, C, F, S) == E_OVERLAP


def test_attention_validation(lib):
    ok = dict(q=E, qs=256, c=_c(), table=F, width=2, lens=G, start=H, total=5, heads=4, batch=2, max_q=5, max_len=32,
              scale=0.1, t=0, out=9 << 36, ws=None, nws=0, s=S)

    def call(**k):
        return lib.atom_kv4_attention(*{**ok, **k}.values())
    for n in ("q", "table", "lens", "start", "out", "c"):
        assert call(**{n: None}) == E_NULL
    for bad in (dict(heads=5), dict(heads=1), dict(heads=0), dict(total=0), dict(batch=0), dict(max_q=0), dict(max_len=0),
                dict(width=0), dict(width=1 << 27), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(t=2), dict(qs=248), dict(c=_c(dim=32)), dict(max_len=(1 << 30) + 1)):
        assert call(**bad) == E_SHAPE, bad
    assert call(q=E + 2) == call(qs=260) == call(table=F + 2) == call(out=(9 << 36) + 4) == E_ALIGN
    assert call(out=E) == call(out=A) == call(out=H) == E_OVERLAP
    need = lib.atom_kv4_attention_workspace_bytes(5, 4, 2, 64, 2, 1, 4096)
    assert need > 0
    more = dict(max_q=1, max_len=4096, width=256)
    assert call(ws=(10 << 36) + 4, nws=need, **more) == E_ALIGN
    assert call(ws=A, nws=need, **more) == E_OVERLAP
    assert lib.atom_kv4_attention_workspace_bytes(5, 3, 2, 64, 2, 1, 4096) == -E_SHAPE
    assert lib.atom_kv4_attention_workspace_bytes(1 << 20, 64, 8, 128, 256, 1 << 20, 4096) == -E_SHAPE   # 2^27 workgroups
    assert lib.atom_kv4_attention_workspace_bytes(1 << 20, 64, 8, 128, 256, 1 << 12, 4096) >= 0
    assert lib.atom_kv4_attention_workspace_bytes(1, 2, 2, 64, 1, 1, 100) == 0
    with pytest.raises(bq.AtomError):
        bq.atom_kv4_attention_workspace_bytes(5, 3, 2, 64, 2, 1, 4096)


class _NoLaunch:
    """The loaded library with every entry point that would enqueue work replaced by a failure."""

    def __init__(self, lib):
        self._lib = lib

    def __getattr__(self, name):
        if name.endswith(("_bytes", "strerror")):
            return getattr(self._lib, name)

        def fail(*a):
            raise AssertionError(f"{name} was called with arguments the binding should have refused")
        return fail


def test_binding_refusals(lib, monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(bq, "_LIB", _NoLaunch(lib))
    z, f16, b16, f32, i8, u8, i32, i64 = (torch.zeros, torch.float16, torch.bfloat16, torch.float32, torch.int8,
                                          torch.uint8, torch.int32, torch.int64)
    X, Wq, sw = z((4, 200), dtype=f16), z((6, 256), dtype=i8), z((6,), dtype=f32)
    Xq, sx = z((4, 256), dtype=i8), z((4,), dtype=f32)
    cache = bq.kv4_cache(3, 16, 2, 64, device="cpu")
    K, slots = z((5, 2, 64), dtype=f16), z((5,), dtype=i64)
    Q, table, lens, start = z((5, 4, 64), dtype=f16), z((2, 3), dtype=i32), z((2,), dtype=i32), z((3,), dtype=i32)
    shape = [
        lambda: bq.atom_quantize_w8a8(X, Xq=z((4, 200), dtype=i8)),
        lambda: bq.atom_quantize_w8a8(X, sx=z((5,), dtype=f32)),
        lambda: bq.atom_quantize_w8a8(X[0]),
        lambda: bq.atom_gemm_w8a8(Xq, sx, Wq, sw, 300),
        lambda: bq.atom_gemm_w8a8(Xq, z((3,), dtype=f32), Wq, sw, 200),
        lambda: bq.atom_gemm_w8a8(Xq, sx, Wq, sw, 200, bias=z((4,), dtype=f16)),
        lambda: bq.atom_gemm_w8a8(Xq, sx, Wq, sw, 200, Y=z((6, 4), dtype=f16)),
        lambda: bq.atom_gemm_w8a8(Xq, sx, Wq, sw, 200, workspace=z((8, 8), dtype=u8)),
        lambda: bq.linear_w8a8(X, z((6, 200), dtype=i8), sw),
        lambda: bq.linear_w8a8(X, Wq, z((7,), dtype=f32)),
        lambda: bq.linear_w8a8(z((8, 200), dtype=f16), Wq, sw, workspace=z((16,), dtype=u8)),
        lambda: bq.atom_kv4_append(K, K[:4], slots, cache),
        lambda: bq.atom_kv4_append(K, K, z((5, 1), dtype=i64), cache),
        lambda: bq.atom_kv4_append(z((5, 2, 32), dtype=f16), K, slots, cache),
        lambda: bq.atom_kv4_append(K, K, slots, cache._replace(v=cache.k)),
        lambda: bq.atom_kv4_append(K, K, slots, cache._replace(k_par=cache.k_par[:2])),
        lambda: bq.atom_kv4_append(K, K, slots, bq.kv4_cache(3, 24, 2, 64, device="cpu")),
        lambda: bq.atom_kv4_append(K, K, slots, bq.kv4_cache(3, 16, 2, 96, device="cpu")),
        lambda: bq.atom_kv4_read(cache, slots, K=z((4, 2, 64), dtype=f16)),
        lambda: bq.atom_kv4_attention(Q[0], cache, table, lens, start),
        lambda: bq.atom_kv4_attention(z((5, 4, 128), dtype=f16), cache, table, lens, start),
        lambda: bq.atom_kv4_attention(z((5, 3, 64), dtype=f16), cache, table, lens, start),
        lambda: bq.atom_kv4_attention(Q, cache, table, lens, start[:2]),
        lambda: bq.atom_kv4_attention(Q, cache, table, z((3,), dtype=i32), start),
        lambda: bq.atom_kv4_attention(Q, cache, table[0], lens, start),
        lambda: bq.atom_kv4_attention(Q, cache, table, lens, start, out=z((5, 4, 32), dtype=f16)),
        lambda: bq.atom_kv4_attention(Q, cache, table, lens, start, workspace=z((4, 4), dtype=u8)),
    ]
    for i, call in enumerate(shape):
        with pytest.raises(bq.AtomError, match="shape|-D"):
            print(i)
            call()
    kind = [
        lambda: bq.atom_quantize_w8a8(X.float()),
        lambda: bq.linear_w8a8(X, Wq, sw, bias=z((6,), dtype=b16)),
        lambda: bq.linear_w8a8(X, Wq.view(u8), sw),
        lambda: bq.linear_w8a8(X, Wq, sw.half()),
        lambda: bq.atom_gemm_w8a8(Xq, sx, Wq, sw, 200, dtype=f32),
        lambda: bq.atom_kv4_append(K, K.bfloat16(), slots, cache),
        lambda: bq.atom_kv4_append(K, K, slots.int(), cache),
        lambda: bq.atom_kv4_read(cache, slots, dtype=f32),
        lambda: bq.atom_kv4_attention(Q, cache, table.long(), lens, start),
        lambda: bq.atom_kv4_attention(Q, cache, table, lens, start, out=z((5, 4, 64), dtype=b16)),
    ]
    for call in kind:
        with pytest.raises(bq.AtomError, match="must be"):
            call()
    with pytest.raises(bq.AtomError, match="agree"):
        bq.atom_gemm_w8a8(Xq, sx, Wq, sw, 200, bias=z((6,), dtype=b16), dtype=f16)
    with pytest.raises(bq.AtomError, match="four tensors"):
        bq.atom_kv4_append(K, K, slots, cache[:3])
    # rows may lie apart but not their elements, and no two rows may share memory
    cols = z((200, 4), dtype=f16).t()
    for call in (lambda: bq.linear_w8a8(cols, Wq, sw), lambda: bq.linear_w8a8(X[:1].expand(4, 200), Wq, sw),
                 lambda: bq.atom_kv4_append(z((5, 64, 2), dtype=f16).transpose(1, 2), K, slots, cache),
                 lambda: bq.atom_kv4_attention(z((4, 5, 64), dtype=f16).transpose(0, 1), cache, table, lens, start)):
        with pytest.raises(bq.AtomError, match="contiguous|ROCm device"):
            call()
    # well-formed host tensors get as far as the device check
    for call in (lambda: bq.atom_quantize_w8a8(X), lambda: bq.linear_w8a8(X, Wq, sw),
                 lambda: bq.atom_gemm_w8a8(Xq, sx, Wq, sw, 200), lambda: bq.atom_kv4_append(K, K, slots, cache),
                 lambda: bq.atom_kv4_read(cache, slots), lambda: bq.atom_kv4_attention(Q, cache, table, lens, start)):
        with pytest.raises(bq.AtomError, match="ROCm device"):
            call()
    assert ctypes.sizeof(kv4._CCache) == 48
