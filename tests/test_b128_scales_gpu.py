"""Products whose operands' scales are far apart in size, or whose product of two is below fp32's normal
numbers or above them.

A block's term is its sum T times the product sA sB, which is rounded to fp32 first.  Tolerance: that of the
other products, 1e-5 sum |a b| + 1 step of fp32 (test_b128_gpu.py; the sum counts the scales), and what
a product below 2^-126 loses: half of fp32's least step, 2^-150, times sum |a b| of the codes.  Where a
product is 2^128 or more, the result is no number."""

import numpy as np
import pytest
import torch

from grouped_gemm_epilogues_gb300 import binding as gge
from oracle import b128, formats

from helpers import dec

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def _codes(rows, cols, seed):
    """Random codes of either sign."""
    g = torch.Generator().manual_seed(seed)
    size = torch.randint(1, 127, (rows, cols), generator=g)
    c = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.uint8)
    c[:, :cols] = size + 128 * torch.randint(0, 2, (rows, cols), generator=g)
    return c.to(DEV)


def _product(ca, sa, cb, sb, k, b_rows, tile, flags=0):
    """D of codes and scales, what it should be, and its tolerance."""
    A = gge.B128Tensor(ca[:, :k].view(torch.float8_e4m3fn), sa.to(DEV))
    B = gge.B128Tensor(cb[:, :k].view(torch.float8_e4m3fn), sb.to(DEV), b_rows)
    D = torch.full((ca.shape[0], cb.shape[0]), 7.0, device=DEV)
    gge.gge_gemm_b128(A, B, D=D, config=gge.make_config(tile_n=tile, flags=flags))
    assert gge.gge_read_device_status(DEV)[0] == "GGE_OK"
    ca, cb = ca[:, :k].cpu().numpy(), cb[:, :k].cpu().numpy()
    a, b = b128.decode(ca, sa.numpy(), "e4m3"), b128.decode(cb, sb.numpy(), "e4m3", b_rows)
    codes = np.abs(formats.decode(ca, formats.E4M3)) @ np.abs(formats.decode(cb, formats.E4M3)).T
    return dec(D), a @ b.T, 1e-5 * (np.abs(a) @ np.abs(b).T) + 2.0 ** -150 * codes


def _check(got, want, tol):
    r = formats.round_to(want, formats.F32)
    worst = np.abs(got - r) / (tol + formats.quantum(r, formats.F32))
    assert worst.max() <= 1.0, worst.max()


# (sA, sB): within the range, at its ends, and with a product below the normal numbers
SIZES = [(1e-25, 1e25), (3e-20, 3e-20), (2.0 ** -126, 1.0), (1e20, 1e10), (1e-40, 1e20), (1e20, 1e-40),
         (1e-30, 1e-12), (1e-12, 1e-30), (2.0 ** -126, 2.0 ** -15), (2.0 ** -20, 2.0 ** -126), (1e-30, 1e-30)]
TILES = [(256, 0), (128, 32), (64, 32), (64, 0)]


@pytest.mark.parametrize("tile,flags", TILES)
@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("sa,sb", SIZES)
def test_scales_of_all_sizes(tile, flags, b_rows, sa, sb):
    m, n, k = 150, 264, 700
    blocks = 6
    g = torch.Generator().manual_seed(int(tile + b_rows))
    a = sa * torch.exp2(torch.randint(0, 2, (m, blocks), generator=g).float())
    b = sb * torch.exp2(torch.randint(0, 2, (n if b_rows == 1 else 3, blocks), generator=g).float())
    _check(*_product(_codes(m, k, 1), a, _codes(n, k, 2), b, k, b_rows, tile, flags))


@pytest.mark.parametrize("tile,flags", TILES)
@pytest.mark.parametrize("b_rows", [1, 128])
def test_sizes_side_by_side(tile, flags, b_rows):
    """Every row and column (or block of them) has another size, blocks of K differ, some scales are
    zero, and more blocks than the ring of scales holds at a time."""
    m, n, k = 150, 264, 2500
    blocks = 20
    sa = torch.exp2(torch.linspace(-126, 40, m)).reshape(m, 1).repeat(1, blocks)
    sa[:, 5], sa[:, 6], sa[20:30, 9] = sa[:, 5] * 2.0 ** -3, 0.0, 0.0
    rows = n if b_rows == 1 else 3
    sb = torch.exp2(torch.linspace(-30, 20, rows)).reshape(rows, 1).repeat(1, blocks)
    sb[:, 13], sb[0, 11] = sb[:, 13] * 2.0 ** 5, 0.0
    _check(*_product(_codes(m, k, 3), sa, _codes(n, k, 4), sb, k, b_rows, tile, flags))


@pytest.mark.parametrize("tile,flags", TILES)
@pytest.mark.parametrize("b_rows", [1, 128])
def test_zeros_and_scales_that_are_not_finite(tile, flags, b_rows):
    """A row of zeros under its least scale gives zeros; a NaN or infinite scale, or one whose product
    with B's is too large, spoils its row and no other."""
    m, n, k = 70, 136, 300
    ca, cb = _codes(m, k, 5), _codes(n, k, 6)
    ca[3] = 0
    sa, sb = torch.ones(m, 3), torch.full((n if b_rows == 1 else 2, 3), 1e15)
    sa[3], sa[4] = 2.0 ** -126, 2.0 ** -126
    sa[40, 1], sa[41, 2], sa[42, 0] = float("nan"), float("inf"), 1e30
    with np.errstate(invalid="ignore"):
        got, want, tol = _product(ca, sa, cb, sb, k, b_rows, tile, flags)
    ok = [i for i in range(m) if i not in (40, 41, 42)]
    _check(got[ok], want[ok], tol[ok])
    assert not got[3].any() and not np.isfinite(got[40:43]).any()
