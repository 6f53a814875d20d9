"""Values that lie exactly on a border of two codes or blocks although the norm is no power of two (needs an MI355X).

A row of +-c over K elements has the sum of squares K c^2, exact in 64 bits, so the mean is c^2, the root c and y = c w / c = w,
each step without a rounding (eps is far below the mean's last place, or in it, which the oracle's 64 bits see as the kernel's
do).  Multiplying by 1 / K or by 1 / c instead leaves such values a step of 2^-53 beside the border."""
import numpy as np
import pytest

from test_gpu_norm import TYPES, _gpu, bq, check, say  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

MX = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 1.0, 2.0, 4.0, 0.5, 3.0, 6.0, 7.0, 1.5)
INT8 = (127.0, 0.5, 1.5, 2.5, 3.5, 62.5, 63.5, 31.5, 16.5, 126.5, 100.0)      # the scale is 1


def rows(K, t):
    sign = torch.where(torch.arange(K) % 2 == 0, 1.0, -1.0)
    return (torch.tensor([1.0, 3.0, 7.0, 11.0, 13.0, 49.0, 0.375, 23.0, 98.0, 107.0])[:, None] * sign).to(t).cuda()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [33, 49, 98, 103, 161, 196, 256, 300, 1155, 4097])
def test_ties_of_any_norm(K, dtype):
    say(f"[norm ties] K={K} {dtype}")
    t = TYPES[dtype]
    x = rows(K, t)
    for border in (MX, INT8):
        w = torch.from_numpy(np.resize(np.array(border + tuple(-b for b in border)), K)).to(t).cuda()
        for eps in (1e-40, 1e-13):
            check(x, w, eps)
            check(x, w, eps, torch.zeros_like(x))


@pytest.mark.parametrize("dtype", TYPES)
def test_a_block_whose_largest_is_a_power_of_two(dtype):
    """The block's exponent is the formula's: 4 is 4 of 2^0, not of 2^-1."""
    t = TYPES[dtype]
    x = rows(256, t)
    for top in (4.0, 2.0, 1.0, 0.5):
        w = (torch.tensor([1.0, 0.25, 0.75, 0.5] * 64) * top).to(t).cuda()
        check(x, w, 1e-40)
        check(x, w, 1e-14)


def test_ties_of_rows_apart_and_in_place():
    """The sum in place of one of its terms, rows that lie apart and begin anywhere: the codes of contiguous rows."""
    t = torch.float16
    K = 300
    w = torch.from_numpy(np.resize(np.array(MX + INT8), K)).to(t).cuda()
    h = rows(K, t)
    r = torch.ones_like(h)
    x = h - 1
    for call in (bq.atom_rmsnorm_w8a8, bq.atom_rmsnorm_mxfp4):
        want = call(h, w, 1e-40)
        check(h, w, 1e-40)
        for first in (0, 8, 3):
            wide = torch.full((len(h), 400), 7.0, dtype=t, device="cuda")
            apart = wide[:, first:first + K]
            apart.copy_(x)
            for place in ("none", "residual", "x"):
                a, b = apart.clone() if place == "x" else apart, r.clone()
                H = {"none": None, "residual": b, "x": a}[place]
                Xq, sx, H = call(a, w, 1e-40, residual=b, H=H)
                torch.testing.assert_close(H, h, rtol=0, atol=0)
                torch.testing.assert_close(Xq, want[0], rtol=0, atol=0)
                torch.testing.assert_close(sx, want[1], rtol=0, atol=0)
            Xq, sx, _ = call(apart, w, 1e-40, residual=r, H=apart)
            torch.testing.assert_close(Xq, want[0], rtol=0, atol=0)
            assert torch.equal(apart, h) and torch.all(wide[:, :first] == 7) and torch.all(wide[:, first + K:] == 7)
