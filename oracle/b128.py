"""8-bit codes with a scale for each block of 128, and layer norm, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

A block is 128 columns of one row, or of 128 rows.  scale = max(max|x| * (1 / top),
2^-126), code = x * (1 / scale) rounded to the format, at most top in size (448 for
e4m3, 57344 for e5m2); both products and the reciprocal are fp32 operations, as the
definition says.  A block with an infinity or a NaN has a NaN scale.
"""

import numpy as np

from . import formats

BLOCK = 128
TOP = {"e4m3": 448.0, "e5m2": 57344.0}


def _blocks(x, block_rows):
    """(row blocks, column blocks, block_rows, 128), padded with zeros."""
    rows, cols = x.shape
    nr, nc = -(-rows // block_rows), -(-cols // BLOCK)
    full = np.zeros((nr * block_rows, nc * BLOCK))
    full[:rows, :cols] = x
    return full.reshape(nr, block_rows, nc, BLOCK).transpose(0, 2, 1, 3)


def spread(scales, rows, cols, block_rows):
    """One scale a value."""
    return np.repeat(np.repeat(scales, block_rows, 0)[:rows], BLOCK, 1)[:, :cols]


def quantise(x, fmt="e4m3", block_rows=1):
    """x (rows, cols) float64 of fp32 values -> (values, scales (row blocks, column blocks)),
    both float64; `values` are the numbers that the codes stand for."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    f = np.float32
    b = _blocks(x, block_rows)
    bad = ~np.isfinite(b).all((2, 3))
    amax = np.abs(np.where(bad[:, :, None, None], 0.0, b)).max((2, 3)).astype(f)
    scale = np.maximum(amax * (f(1.0) / f(TOP[fmt])), f(2.0 ** -126))
    inv = f(1.0) / scale
    fin = np.where(spread(bad, rows, cols, block_rows), 0.0, x)
    scaled = (fin.astype(f) * spread(inv, rows, cols, block_rows)).astype(np.float64)
    code = formats.round_to(np.clip(scaled, -TOP[fmt], TOP[fmt]), formats.BY_NAME[fmt])
    scale = np.where(bad, np.nan, scale.astype(np.float64))
    return code * spread(scale, rows, cols, block_rows), scale


def decode(codes, scales, fmt="e4m3", block_rows=1):
    """The numbers that stored codes (bytes) and scales stand for."""
    c = formats.decode(codes, formats.BY_NAME[fmt])
    with np.errstate(invalid="ignore"):
        return c * spread(np.asarray(scales, dtype=np.float64), *c.shape, block_rows)


def off_codes(got, scales, want, tol, fmt="e4m3"):
    """How far quantised numbers (blocks of a row) are from `want`, which the code rounds from
    within `tol`, in units of what is allowed: half a step of the code's grid and tol; and how far
    the scales are from max|want| / top, in units of the same tol (and fp32's rounding)."""
    rows, cols = want.shape
    f = formats.BY_NAME[fmt]
    unit = spread(np.asarray(scales, dtype=np.float64), rows, cols, 1)
    scaled = np.abs(want) / unit
    half = formats.quantum(np.minimum(scaled, TOP[fmt]), f) / 2
    over = np.maximum(scaled - TOP[fmt], 0.0)
    value = np.abs(got - want) / (unit * (half + over) + tol + 2.0 ** -22 * np.abs(want))
    amax = np.abs(_blocks(want, 1)).max((2, 3))
    slack = _blocks(np.broadcast_to(tol, want.shape), 1).max((2, 3)) + 2.0 ** -22 * amax + 2.0 ** -126 * TOP[fmt]
    scale = np.abs(np.asarray(scales, dtype=np.float64) * TOP[fmt] - amax) / slack
    return float(value.max()), float(scale.max())


def layernorm(x, w, b, eps, residual=None, h_fmt=None):
    """(h, mean, rstd, y): h rounded to h_fmt where a residual is added, the rest unrounded."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = formats.round_to(h + residual, h_fmt)
    mean = h.mean(1)
    d = h - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    return h, mean, rstd, d * rstd[:, None] * w + b


def layernorm_bwd(dy, h, w, mean, rstd, dh=None):
    """(dx, dw, db) for the saved mean and rstd."""
    rstd = np.asarray(rstd, dtype=np.float64)[:, None]
    n = (h - np.asarray(mean, dtype=np.float64)[:, None]) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdims=True) - n * (g * n).mean(1, keepdims=True))
    return dx if dh is None else dx + dh, (dy * n).sum(0), dy.sum(0)
