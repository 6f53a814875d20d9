"""The MXFP4 product behind the norm, with scratch memory as the layer has it (needs an MI355X): long K is divided there too."""
import pytest

from test_gpu_mxfp4 import _gpu, bq, check_y, make, say, values  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(64, 4096, 8192), (777, 777, 8192), (333, 512, 28672), (200, 260, 4096)])
def test_norm_then_product(M, N, K):
    """The product of the norm's rows with as much scratch as atom_gemm_mxfp4_workspace_bytes says (none for the last shape): by either way
    the same bits, those of the layer on the same rows, and within the sum's steps of fp64."""
    say(f"[mxfp4 chain] {M}x{N}x{K}")
    t = torch.bfloat16
    Wq, sw = bq.atom_quantize_mxfp4(make(N, K, t, 2, 0.02))
    Xq, sx, H = bq.atom_rmsnorm_mxfp4(make(M, K, t, 1), torch.ones(K, dtype=t, device="cuda"), 1e-6, residual=make(M, K, t, 3))
    need = bq.atom_gemm_mxfp4_workspace_bytes(M, N, K)
    assert (need > 0) == (K > 4096)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    Y = bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, K, dtype=t, workspace=ws)
    full = bq.atom_gemm_mxfp4(Xq, sx, Wq, sw, K, dtype=t, workspace=ws, stream=torch.cuda.current_stream())
    torch.testing.assert_close(Y, full, rtol=0, atol=0)
    check_y(Y, values(Xq, sx), values(Wq, sw), None, K, f"{M}x{N}x{K}")
    # what the codes stand for quantizes to the codes again, so the layer multiplies the same operands by the same plan
    X = bq.atom_dequantize_mxfp4(Xq, sx, K, dtype=t)
    if bq.atom_linear_mxfp4_workspace_bytes(M, N, K):
        torch.testing.assert_close(Y, bq.linear_mxfp4(X, Wq, sw), rtol=0, atol=0)
