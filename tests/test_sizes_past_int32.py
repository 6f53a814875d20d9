"""Sizes that do not fit the C ABI's 32-bit arguments are refused, never cut to their low bits (no GPU needed, no kernel is launched)."""
import os

import pytest

import bit_quantized_gemm_amd as bq

torch = pytest.importorskip("torch")
BIG = 1 << 32
E_SHAPE = 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bq.lib_path()):
        pytest.skip("libatom.so not built (python -m bit_quantized_gemm_amd.build)")
    return bq.load_library()


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


def test_size_queries(lib):
    for K in (BIG + 300, -BIG + 300, BIG * BIG + 300):
        assert bq.atom_mxfp4_row_bytes(K) == bq.atom_mxfp4_groups(K) == bq.atom_w8a8_row_bytes(K) == -E_SHAPE
        assert bq.atom_row_bytes(K) < 0 and bq.atom_num_groups(K) < 0
        for query in (bq.atom_gemm_mxfp4_workspace_bytes, bq.atom_linear_mxfp4_workspace_bytes, bq.atom_gemm_w8a8_workspace_bytes,
                      bq.atom_linear_w8a8_workspace_bytes):
            for shape in ((K, 4, 4), (4, K, 4), (4, 4, K)):
                with pytest.raises(bq.AtomError):
                    query(*shape)


def test_calls(lib, monkeypatch):
    """Each of these would pass with its size's low 32 bits."""
    monkeypatch.setattr(bq, "_LIB", _NoLaunch(lib))
    z, u8, i8, i32, f32 = torch.zeros, torch.uint8, torch.int8, torch.int32, torch.float32
    Xq, sx, Wq, sw = z((4, 256), dtype=u8), z((2, 4, 8), dtype=u8), z((6, 256), dtype=u8), z((2, 6, 8), dtype=u8)
    lens, table, pool, done = z(5, dtype=i32), z((5, 3), dtype=i32), bq.kv4_pool(9, device="cpu"), z(5, dtype=torch.bool)
    tall = z(1, dtype=torch.float16).expand(BIG + 4).unsqueeze(1)          # (a view of one element)
    one = z((1, 128), dtype=u8), z((1, 1, 8), dtype=u8)
    calls = [
        lambda: bq.atom_dequantize_mxfp4(Xq, sx, BIG + 300),
        lambda: bq.atom_dequantize_w8a8(z((4, 384), dtype=i8), z(4, dtype=f32), BIG + 300),
        lambda: bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, BIG + 300),
        lambda: bq.linear_mxfp4(tall, *one),
        lambda: bq.atom_rmsnorm_mxfp4(tall, z(1, dtype=torch.float16)),
        lambda: bq.atom_rmsnorm_w8a8(tall, z(1, dtype=torch.float16)),
        lambda: bq.atom_quantize_mxfp4(tall),
        lambda: bq.atom_kv4_extend(lens, lens.clone(), table, pool, 16, BIG + 7),
        lambda: bq.atom_kv4_extend(lens, lens.clone(), table, pool, BIG + 16, 7),
        lambda: bq.atom_kv4_extend(lens, lens.clone(), z(1, dtype=i32).expand(BIG + 5).unsqueeze(1), pool, 16, 7),
        lambda: bq.atom_kv4_release(done, lens, table, pool, BIG + 16),
    ]
    for i, call in enumerate(calls):
        print(i)
        with pytest.raises(bq.AtomError, match=r"2\*\*31|status 2"):
            call()
