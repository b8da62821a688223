"""Low-precision linear layer in float64: microscaled formats, RMS norm.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Formats: e4m3 or e2m1 codes along K, a scale per block of 32 (mxfp8, mxfp4:
2^(byte - 127), byte 255 = NaN) or 16 (nvfp4: e4m3, times one fp32 scale a
tensor).  Power-of-two scales are the smallest 2^e, e >= -127, with max|x| <= 2^e
* (448 or 6); nvfp4's are e4m3(min(max(max|x| / (6 t), 2^-9), 448)) and its codes
e2m1(x * (1 / (s t))), in fp32 arithmetic as the definition says.  A block with an
infinity or a NaN is NaN throughout.
"""

import numpy as np

from . import formats

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
TOP = {"mxfp8": 448.0, "mxfp4": 6.0, "nvfp4": 6.0}


def round_e2m1(x):
    """Nearest of the e2m1 values, halfway to the even code, at most 6 in size."""
    a = np.minimum(np.abs(x), 6.0)
    i = np.zeros(a.shape, dtype=np.int64)
    for k in range(7):
        mid = (E2M1[k] + E2M1[k + 1]) / 2
        i += (a > mid) | ((a == mid) & ((k + 1) % 2 == 0))
    return i, np.where(x < 0, -E2M1[i], E2M1[i])


def quantise(x, fmt, t=1.0):
    """x (rows, cols) float64 -> (values, scale bytes (rows, blocks)).  `values` are the
    numbers that the codes stand for (float64)."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    size = BLOCK[fmt]
    nb = -(-cols // size)
    v = np.zeros((rows, nb * size))
    v[:, :cols] = x
    v = v.reshape(rows, nb, size)
    bad = ~np.isfinite(v).all(2)
    v = np.where(bad[:, :, None], 0.0, v)
    amax = np.abs(v).max(2)
    if fmt == "nvfp4":
        f = np.float32
        with np.errstate(over="ignore"):
            want = amax.astype(f) / (f(6.0) * f(t))
        s = formats.round_to(np.clip(want.astype(np.float64), 2.0 ** -9, 448.0), formats.E4M3)
        byte = formats.encode(s, formats.E4M3)
        r = (f(1.0) / (s.astype(f) * f(t)))[:, :, None]
        scaled = (v.astype(f) * r).astype(np.float64)
        unit = (s * float(f(t)))[:, :, None]
    else:
        m, e = np.frexp(amax / TOP[fmt])          # amax / top = m 2^e, m in [0.5, 1)
        e = np.where(m == 0.5, e - 1, e)          # an exact power of two needs no more
        e = np.clip(np.where(amax == 0, -127, e), -127, 127)
        byte = e + 127
        unit = np.ldexp(1.0, e)[:, :, None]
        scaled = v / unit
    if fmt == "mxfp8":
        code = formats.round_to(scaled, formats.E4M3)
    else:
        code = round_e2m1(scaled)[1]
    out = np.where(bad[:, :, None], np.nan, code * unit)
    byte = np.where(bad, 0x7F if fmt == "nvfp4" else 255, byte)
    return out.reshape(rows, -1)[:, :cols], byte.astype(np.uint8)


def scale_offset(row, block, blocks):
    """Byte of the scale of (row, block) among a matrix's scale tiles."""
    tile = (row // 128) * (-(-blocks // 4)) + block // 4
    return tile * 512 + (row % 32) * 16 + (row % 128) // 32 * 4 + block % 4


def scale_bytes(flat, rows, cols, fmt):
    """(rows, blocks) scale bytes out of the tiles `flat`, and the padding of those rows."""
    blocks = -(-cols // BLOCK[fmt])
    r, b = np.meshgrid(np.arange(rows), np.arange(-(-blocks // 4) * 4), indexing="ij")
    got = np.asarray(flat)[scale_offset(r, b, blocks)]
    return got[:, :blocks], got[:, blocks:]


def decode(codes, flat, rows, cols, fmt, t=1.0):
    """The numbers that stored codes (rows, bytes) and scale tiles stand for, as float64."""
    codes = np.asarray(codes, dtype=np.uint8)
    if fmt == "mxfp8":
        c = formats.decode(codes, formats.E4M3)
    else:
        nib = np.stack((codes & 15, codes >> 4), 2).reshape(rows, -1)
        c = np.where(nib & 8, -1.0, 1.0) * E2M1[nib & 7]
    s = scale_bytes(flat, rows, cols, fmt)[0]
    if fmt == "nvfp4":
        unit = formats.decode(s, formats.E4M3) * float(np.float32(t))
    else:
        unit = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    unit = np.repeat(unit, BLOCK[fmt], axis=1)
    return c[:, :cols] * unit[:, :cols]


def rmsnorm(x, w, eps, residual=None, h_fmt=None):
    """(h, inv, y): h rounded to h_fmt where a residual is added, the rest unrounded."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = formats.round_to(h + residual, h_fmt)
    inv = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h, inv, h * inv[:, None] * w


def rmsnorm_bwd(dy, h, w, inv, dh=None):
    """(dx, dw) for the saved inv."""
    g = dy * w
    inv = np.asarray(inv, dtype=np.float64)[:, None]
    dx = inv * (g - h * inv * inv * (g * h).mean(1, keepdims=True))
    return dx if dh is None else dx + dh, (dy * h * inv).sum(0)
