"""Rows that the layer norm's joins of threads and warps could get wrong: an infinity or a NaN in any
place, and one value far from all others where a row begins.

The tolerances are those of test_layernorm_gpu.py, derived there.  What is not finite has none: a row
that holds an infinity or a NaN has no variance, so its rstd, and with it all of its y, is NaN."""

import numpy as np
import pytest
import torch

from grouped_gemm_epilogues_gb300 import binding as gge
from oracle import b128

from test_layernorm_gpu import DEV, EPS, TYPES, _empty, _forward_ref, _near, _numbers, _rand

pytestmark = pytest.mark.gpu
LIES = ("aligned", "alike", "any")   # where rows start against 16 bytes: on them, alike, each elsewhere


def _place(x, lie, spare=8):
    """x's values in rows that lie so, and room for as many results."""
    rows, cols = x.shape
    pitch = cols + spare if lie != "aligned" else (cols + 7) // 8 * 8
    first = 0 if lie == "aligned" else 3
    wide, out = (torch.zeros(rows, pitch, dtype=x.dtype, device=DEV) for _ in range(2))
    wide[:, first:first + cols] = x
    second = first if lie != "any" else 0
    return wide[:, first:first + cols], out[:, second:second + cols]


def _norm(x, w, lie, codes):
    at, y = _place(x, lie)
    rows, cols = x.shape
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    q, h8 = (_empty(rows, cols), _empty(rows, cols)) if codes else (None, None)
    gge.gge_layernorm(at, w, Y=y, Q=q, H8=h8, mean=mean, rstd=rstd, eps=EPS)
    return y, mean, rstd, q, h8


@pytest.mark.parametrize("cols", [1, 7, 200, 256, 777, 1000, 4096, 12288, 16384, 16390])
@pytest.mark.parametrize("lie", LIES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("codes", [False, True])
def test_rows_that_are_not_finite(cols, lie, dtype, codes):
    """Each of +inf, -inf and NaN alone in a row, in the first and later lanes, the first and later
    warps and the last place, clean rows between."""
    bad = [float("inf"), float("-inf"), float("nan")]
    places = sorted({c for c in (0, 5, 8, 100, 255, 300, 2100, 9000, cols - 1) if c < cols})
    rows = 2 * len(bad) * len(places) + 1
    clean = _rand(rows, cols, dtype, 5)
    x, w = clean.clone(), _rand(1, cols, dtype, 6)[0]
    hit = []
    for i, (value, c) in enumerate((v, c) for v in bad for c in places):
        x[2 * i + 1, c] = value
        hit.append(2 * i + 1)
    rest = np.setdiff1d(np.arange(rows), hit)
    y, mean, rstd, q, h8 = _norm(x, w, lie, codes)
    y0, mean0, rstd0, q0, h80 = _norm(clean, w, lie, codes)
    assert torch.isnan(y[hit]).all() and torch.isnan(rstd[hit]).all() and not torch.isfinite(mean[hit]).any()
    assert torch.equal(y[rest], y0[rest]) and torch.equal(mean[rest], mean0[rest]) and torch.equal(rstd[rest], rstd0[rest])
    assert torch.isfinite(y0).all() and torch.isfinite(rstd0).all()
    if codes:
        got, want = _numbers(q), _numbers(q0)
        assert np.isnan(got[hit]).all() and np.array_equal(got[rest], want[rest])
        got, want = _numbers(h8), _numbers(h80)
        assert np.array_equal(got[rest], want[rest])
        # h's codes: the block with the value, and no other
        for i, (_, c) in zip(hit, ((v, c) for v in bad for c in places)):
            block = np.arange(cols) // 128 == c // 128
            assert np.isnan(got[i, block]).all() and np.array_equal(got[i, ~block], want[i, ~block])
    # the backward of such a row is NaN, of the others what it was
    dy = _rand(rows, cols, dtype, 7)
    dx, dx0 = torch.empty_like(dy), torch.empty_like(dy)
    gge.gge_layernorm_bwd(dy, h8 if codes else x, w, mean, rstd, dx)
    gge.gge_layernorm_bwd(dy, h80 if codes else clean, w, mean0, rstd0, dx0)
    assert torch.isnan(dx[hit]).all() and torch.equal(dx[rest], dx0[rest])


@pytest.mark.parametrize("cols", [64, 255, 256, 513, 777, 2056, 4096, 12288, 16384])
@pytest.mark.parametrize("skew", range(8))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("codes", [False, True])
def test_one_value_far_from_the_others(cols, skew, dtype, codes):
    """A channel that stands out, in the first place, the first thread's or the first warp's columns:
    mean, variance and y are as good as for any row."""
    rows = 300
    g = torch.Generator().manual_seed(cols + skew)
    x = torch.randn(rows, cols, generator=g)
    at = [0, 7, 1, 40][skew % 4]
    x[:, at] = torch.exp(torch.empty(rows).uniform_(4.0, 9.0, generator=g))
    x = x.to(dtype).to(DEV)
    wide, out = (torch.zeros(rows, cols + 8 - cols % 8 + 8, dtype=dtype, device=DEV) for _ in range(2))
    wide[:, skew:skew + cols] = x
    w = _rand(1, cols, torch.float32, 3)[0]
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    q = _empty(rows, cols) if codes else None
    y = out[:, skew:skew + cols]
    gge.gge_layernorm(wide[:, skew:skew + cols], w, Y=y, Q=q, mean=mean, rstd=rstd, eps=EPS)
    _, rmean, rrstd, ry, tm, tr, ty = _forward_ref(x, w, None)
    _near(rstd, rrstd, tr, "rstd")
    _near(mean, rmean, tm, "mean")
    _near(y, ry, ty, "y")
    if codes:
        value, scale = b128.off_codes(_numbers(q), q.scales.cpu().numpy(), ry, ty)
        assert value <= 1.0 and scale <= 1.0, (value, scale)
