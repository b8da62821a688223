"""Low-precision operators on matrices of more than 2^31 elements: their last rows have
to be what the same rows give on their own, bit for bit."""

import pytest
import torch

from grouped_gemm_epilogues_gb300 import binding as gge

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
ROWS, TAIL = 2 ** 18 + 1024, 256  # (whole scale tiles of 128 rows)


def _rand(rows, cols, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    return x.normal_(generator=g)


def _same(a, b):
    assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("cols", [8192, 8195])
def test_norm(cols):
    x, r, w = _rand(ROWS, cols, 1), _rand(ROWS, cols, 2), _rand(1, cols, 3)[0]
    h, y, inv = torch.empty_like(x), torch.empty_like(x), torch.empty(ROWS, device=DEV)
    gge.gge_rmsnorm(x, w, Y=y, residual=r, residual_out=h, inv_rms=inv, eps=1e-5)
    t = [v[-TAIL:].clone() for v in (x, r)]
    h2, y2, inv2 = torch.empty_like(t[0]), torch.empty_like(t[0]), torch.empty(TAIL, device=DEV)
    gge.gge_rmsnorm(t[0], w, Y=y2, residual=t[1], residual_out=h2, inv_rms=inv2, eps=1e-5)
    _same(h[-TAIL:], h2)
    _same(inv[-TAIL:], inv2)
    _same(y[-TAIL:], y2)
    del r, y
    dx = torch.empty_like(x)
    gge.gge_rmsnorm_bwd(x, h, w, inv, dx)
    dx2 = torch.empty_like(t[0])
    gge.gge_rmsnorm_bwd(t[0], h2, w, inv[-TAIL:].clone(), dx2)
    _same(dx[-TAIL:], dx2)


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_quantisation(fmt):
    x = _rand(ROWS, 8192, 4)
    tail = x[-TAIL:].clone()
    q, q2 = gge.mx_empty(ROWS, 8192, fmt), gge.mx_empty(TAIL, 8192, fmt)
    values, values2 = torch.empty_like(x), torch.empty_like(tail)
    gge.gge_mx_quantize(x, q, values=values)
    gge.gge_mx_quantize(tail, q2, values=values2)
    _same(q.codes[-TAIL:], q2.codes)
    _same(q.scales.reshape(-1)[-q2.scales.numel():], q2.scales.reshape(-1))
    _same(values[-TAIL:], values2)
    values.fill_(9.0)
    gge.gge_mx_dequantize(q, values)
    _same(values[-TAIL:], values2)
    del q, values
    # the transpose: 8192 rows, whose last columns lie past 2^31 elements
    qt, qt2 = gge.mx_empty(8192, ROWS, fmt), gge.mx_empty(8192, TAIL, fmt)
    gge.gge_mx_quantize(x.t(), qt)
    gge.gge_mx_quantize(tail.t(), qt2)
    per = 1 if fmt == "mxfp8" else 2  # columns a byte
    _same(qt.codes[:, (ROWS - TAIL) // per:ROWS // per], qt2.codes[:, :TAIL // per])


@pytest.mark.parametrize("tile_n", [256, 128, 64])
def test_product(tile_n):
    a, b = _rand(ROWS, 256, 5), _rand(8192, 256, 6)
    qa, qb, qt = gge.mx_empty(ROWS, 256, "nvfp4"), gge.mx_empty(8192, 256, "nvfp4"), gge.mx_empty(TAIL, 256, "nvfp4")
    gge.gge_mx_quantize(a, qa)
    gge.gge_mx_quantize(b, qb)
    gge.gge_mx_quantize(a[-TAIL:].clone(), qt)
    cfg = gge.make_config(tile_n=tile_n)
    c = _rand(ROWS, 8192, 7)
    d, p = torch.empty_like(c), torch.empty_like(c)
    gge.gge_gemm_mx(qa, qb, D=d, PostAct=p, C=c, beta=0.5, act="silu", config=cfg)
    d2 = torch.empty(TAIL, 8192, dtype=c.dtype, device=DEV)
    p2 = torch.empty_like(d2)
    gge.gge_gemm_mx(qt, qb, D=d2, PostAct=p2, C=c[-TAIL:].clone(), beta=0.5, act="silu", config=cfg)
    _same(d[-TAIL:], d2)
    _same(p[-TAIL:], p2)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp8"])
def test_norm_of_one_row_past_2_30_columns(fmt):
    """nvfp4 has a scale word every 64 columns: twice as many a row as the other formats.  The
    codes, scales and values are what gge_mx_quantize makes of the same fp32 y."""
    cols = 2 ** 30 + 1077
    g = torch.Generator(device=DEV).manual_seed(8)
    x = torch.empty(1, cols, device=DEV).normal_(generator=g)
    w = _rand(1, cols, 9)[0]
    t = torch.tensor([2.0 ** -9], device=DEV) if fmt == "nvfp4" else None
    y, inv = torch.full_like(x, 9.0), torch.zeros(1, device=DEV)
    values = torch.full((1, cols), 9.0, dtype=torch.bfloat16, device=DEV)
    q, q2 = (gge.mx_empty(1, cols, fmt, device=DEV, tensor_scale=t) for _ in range(2))
    for z in (q, q2):
        z.codes.fill_(0xA5)
        z.scales.fill_(0xA5)
    gge.gge_rmsnorm(x, w, Y=y, Q=q, values=values, inv_rms=inv, eps=1e-5)
    for at in (0, cols // 2, cols - 4096):
        # two products in fp32, as the kernel takes them
        _same(y[:, at:at + 4096], x[:, at:at + 4096] * inv * w[at:at + 4096].float())
    # (a thread adds up 2^20 squares one after the other: 2^-4 at most, about 2^-14 in fact)
    assert abs(float(inv) - float(x.double().square().mean() + 1e-5) ** -0.5) < 2.0 ** -4
    del x, w
    values2 = torch.empty_like(values)
    gge.gge_mx_quantize(y, q2, values=values2)
    _same(q.codes, q2.codes)
    _same(q.scales.view(-1, 32, 16)[:, 0, :4], q2.scales.view(-1, 32, 16)[:, 0, :4])
    _same(values, values2)
