"""Layer norm with the residual's addition, its 8-bit outputs and its backward, on the GPU
against the float64 oracle.

Tolerances.  A lane adds up at most 32 values one after the other (a row of more than 16384
columns: 40), then five steps join a warp's lanes and five the warps: an error of at most N 2^-24
of the sum of sizes, N = 64.  So the mean is off by N 2^-24 mean|h|, the variance by the same of
itself and the square of the mean's error (differences from a mean are taken), rstd by half of
that and 2^-24.  y = (h - mean) rstd w + b follows: relative errors of the two factors, the mean's
error times rstd w, and three roundings.  Outputs are rounded once more: one spacing of their
type.  The backward's sums cancel, so their bounds are relative to the sums of the sizes."""

import numpy as np
import pytest
import torch

from grouped_gemm_epilogues_gb300 import binding as gge
from oracle import b128, formats

from helpers import FMT, dec

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
EPS = 1e-5
N = 64 * 2.0 ** -24
TYPES = (torch.bfloat16, torch.float16, torch.float32)


def _rand(rows, cols, dtype, seed, offset=0, shift=0.0):
    """A (rows, cols) device matrix; `offset` elements into wider rows (any alignment)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols + offset, generator=g) * torch.exp(0.5 * torch.randn(cols + offset, generator=g))
    return (x + shift).to(dtype).to(DEV)[:, offset:]


def _empty(rows, cols, fmt=torch.float8_e4m3fn):
    q = gge.b128_empty(rows, cols, 1, fmt, DEV)
    q.codes.view(torch.uint8).fill_(0xA5)
    q.scales.fill_(float("nan"))
    return q


def _numbers(q):
    fmt = "e5m2" if q.dtype == torch.float8_e5m2 else "e4m3"
    return b128.decode(q.codes.contiguous().view(torch.uint8).cpu().numpy(), q.scales.cpu().numpy(), fmt)


def _forward_ref(x, w, b, r=None):
    """The oracle's numbers and the tolerances of mean, rstd and y."""
    dtype = x.dtype
    wn = dec(w) if w is not None else 1.0
    bn = dec(b) if b is not None else 0.0
    h, mean, rstd, y = b128.layernorm(dec(x), wn, bn, EPS, dec(r) if r is not None else None, FMT[dtype])
    off = N * np.abs(h).mean(1)
    d = h - mean[:, None]
    # var's error: its own sum's, and the mean's, squared and as rounding of each difference
    var = (d * d).mean(1)
    dvar = N * var + off ** 2 + 2 * np.abs(d).mean(1) * 2.0 ** -24 * np.abs(h).max(1)
    rel = 0.5 * dvar * rstd ** 2 + 2.0 ** -23
    tol_y = (off[:, None] * rstd[:, None] + (rel[:, None] + 2.0 ** -22) * np.abs(d) * rstd[:, None] +
             2.0 ** -24 * np.abs(h) * rstd[:, None]) * np.abs(wn) + 2.0 ** -23 * (np.abs(y) + np.abs(bn))
    return h, mean, rstd, y, off + 2.0 ** -24 * np.abs(mean), rel * rstd, tol_y


def _near(got, ref, tol, what):
    fmt = FMT[got.dtype]
    g = dec(got)
    assert np.isfinite(g).all(), what
    worst = np.max(np.abs(g - ref) / (tol + formats.quantum(ref, fmt))) if g.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the tolerance"


SHAPES = [(1, 1), (1, 8), (2, 7), (3, 64), (5, 255), (4, 256), (7, 257), (300, 513), (9, 2049), (160, 4096),
          (2, 8192), (700, 1000), (3, 16383), (2, 16384), (3, 16385), (2, 40001)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("offset", [0, 3])
def test_forward(rows, cols, dtype, residual, offset):
    x, w, b = _rand(rows, cols, dtype, 1, offset), _rand(1, cols, dtype, 2)[0], _rand(1, cols, dtype, 12)[0]
    r = _rand(rows, cols, dtype, 3, offset) if residual else None
    y = torch.full((rows, cols + offset), 9.0, dtype=dtype, device=DEV)
    h = torch.full((rows, cols + offset), 9.0, dtype=dtype, device=DEV) if residual else None
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    gge.gge_layernorm(x, w, b, Y=y[:, offset:], residual=r, residual_out=h[:, offset:] if residual else None,
                      mean=mean, rstd=rstd, eps=EPS)
    rh, rmean, rrstd, ry, tm, tr, ty = _forward_ref(x, w, b, r)
    assert (y[:, :offset] == 9.0).all()
    if residual:
        assert np.array_equal(dec(h[:, offset:]), rh)
        assert (h[:, :offset] == 9.0).all()
    _near(mean, rmean, tm, "mean")
    _near(rstd, rrstd, tr, "rstd")
    _near(y[:, offset:], ry, ty, "y")


@pytest.mark.parametrize("rows,cols", [(4, 300), (40, 4096), (3, 16390)])
@pytest.mark.parametrize("shift", [30.0, 1000.0, -20000.0])
def test_a_large_mean_costs_no_variance(rows, cols, shift):
    """fp32 rows whose mean is far above their spread."""
    x = _rand(rows, cols, torch.float32, 1, shift=shift)
    mean, rstd, y = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV), torch.empty_like(x)
    gge.gge_layernorm(x, Y=y, mean=mean, rstd=rstd, eps=EPS)
    _, rmean, rrstd, ry, tm, tr, ty = _forward_ref(x, None, None)
    _near(mean, rmean, tm, "mean")
    _near(rstd, rrstd, tr, "rstd")
    _near(y, ry, ty, "y")


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("offset", [0, 1])
def test_without_weight_or_bias(weight, bias, offset):
    for cols in (513, 16500):
        x = _rand(70, cols, torch.bfloat16, 4, offset)
        w = _rand(1, cols, torch.float32, 5)[0] if weight else None
        b = _rand(1, cols, torch.float16, 6)[0] if bias else None
        y, y2 = torch.empty(70, cols, dtype=torch.bfloat16, device=DEV), _rand(70, cols, torch.bfloat16, 7, offset)
        for out in (y, y2):
            gge.gge_layernorm(x, w, b, Y=out, eps=EPS)
            _, _, _, ry, _, _, ty = _forward_ref(x, w, b)
            _near(out, ry, ty, "y")


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 64), (5, 255), (7, 300), (300, 513), (160, 4096), (9, 2056),
                                       (2, 16384), (3, 16385)])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("fmt", [torch.float8_e4m3fn, torch.float8_e5m2])
def test_codes(rows, cols, offset, fmt):
    """Codes of y round from within its tolerance; codes of h are exactly its quantisation; what
    lies beside a row's codes is left."""
    dtype = TYPES[cols % 3]
    x, r, w = _rand(rows, cols, dtype, 4, offset), _rand(rows, cols, dtype, 5, offset), _rand(1, cols, torch.float32, 6)[0]
    b = _rand(1, cols, torch.float32, 16)[0]
    buf = torch.full((rows, cols // 16 * 16 + 32), 0xA5, dtype=torch.uint8, device=DEV)
    q = gge.B128Tensor(buf[:, :cols].view(fmt), torch.full(((cols + 127) // 128, rows), float("nan"), device=DEV).t())
    h8 = _empty(rows, cols)
    h = torch.empty(rows, cols, dtype=dtype, device=DEV)
    vals = torch.full((rows, cols + offset), 9.0, dtype=torch.float32, device=DEV)
    gge.gge_layernorm(x, w, b, residual=r, residual_out=h, Q=q, values=vals[:, offset:], H8=h8, eps=EPS)
    rh, _, _, ry, _, _, ty = _forward_ref(x, w, b, r)
    assert np.array_equal(dec(h), rh)
    got = _numbers(q)
    assert np.array_equal(dec(vals[:, offset:]), formats.round_to(got, formats.F32))
    assert (vals[:, :offset] == 9.0).all() and (buf[:, cols:] == 0xA5).all()
    value, scale = b128.off_codes(got, q.scales.cpu().numpy(), ry, ty, "e5m2" if fmt == torch.float8_e5m2 else "e4m3")
    assert value <= 1.0 and scale <= 1.0, (value, scale)
    want, scales = b128.quantise(rh)
    assert np.array_equal(_numbers(h8), want) and np.array_equal(h8.scales.cpu().numpy(), scales)


def test_codes_are_quantise_of_the_norm():
    """The fused output equals gge_b128_quantize of the fp32 y."""
    x, w = _rand(40, 1000, torch.float32, 7), _rand(1, 1000, torch.float32, 8)[0]
    y, q, q2 = torch.empty_like(x), _empty(40, 1000), _empty(40, 1000)
    gge.gge_layernorm(x, w, Y=y, Q=q, eps=EPS)
    gge.gge_b128_quantize(y, q2)
    assert torch.equal(q.codes.view(torch.uint8), q2.codes.view(torch.uint8)) and torch.equal(q.scales, q2.scales)


def test_forward_in_place_and_not_finite():
    """residual_out over the residual; an infinite value and a NaN stay in their rows."""
    x, r, w = _rand(50, 777, torch.bfloat16, 9), _rand(50, 777, torch.bfloat16, 10), _rand(1, 777, torch.bfloat16, 11)[0]
    x[7, 5], x[8, 6] = float("inf"), float("nan")
    rx, rr = x.clone(), r.clone()
    y, q = torch.empty(50, 777, dtype=torch.bfloat16, device=DEV), _empty(50, 777)
    gge.gge_layernorm(x, w, Y=y, residual=r, residual_out=r, Q=q, eps=EPS)
    ok = np.setdiff1d(np.arange(50), [7, 8])
    h, _, _, ry, _, _, ty = _forward_ref(rx[ok], w, None, rr[ok])
    assert np.array_equal(dec(r)[ok], h)
    _near(y[ok], ry, ty, "y")
    assert torch.isnan(y[[7, 8]]).all()
    got = _numbers(q)
    assert np.isnan(got[[7, 8]]).all() and np.isfinite(got[ok]).all()


def test_constant_rows():
    """No variance: rstd is 1 / sqrt(eps) and y the bias."""
    x = torch.full((5, 300), 3.0, device=DEV)
    b = _rand(1, 300, torch.float32, 1)[0]
    y, rstd = torch.empty_like(x), torch.empty(5, device=DEV)
    gge.gge_layernorm(x, None, b, Y=y, rstd=rstd, eps=1e-6)
    assert torch.allclose(rstd, torch.full_like(rstd, 1e3), rtol=1e-6) and torch.equal(y, b.expand(5, 300))


# ----------------------------------------------------------------- backward

def _backward(rows, cols, dtype, offset, with_dh, h8=None, weight=True, seed=20, config=(True, True), shift=0.5):
    dy, w = _rand(rows, cols, dtype, seed, offset), _rand(1, cols, dtype, seed + 1)[0] if weight else None
    h = _rand(rows, cols, dtype, seed + 2, offset, shift=shift)
    dh = _rand(rows, cols, dtype, seed + 3, offset) if with_dh else None
    if h8 is not None:
        H = _empty(rows, cols, h8)
        gge.gge_b128_quantize(h, H)
        hn = formats.round_to(_numbers(H), formats.F32)
    else:
        H, hn = h, dec(h)
    _, mean, rstd, _ = b128.layernorm(dec(h), 1.0, 0.0, EPS)
    mean, rstd = (torch.tensor(v, dtype=torch.float32, device=DEV) for v in (mean, rstd))
    dx = torch.full((rows, cols + offset), 9.0, dtype=dtype, device=DEV)
    dw, db = (torch.full((cols,), float("nan"), device=DEV) if want else None for want in config)
    gge.gge_layernorm_bwd(dy, H, w, mean, rstd, dx[:, offset:], dW=dw, dB=db, dH=dh)
    assert (dx[:, :offset] == 9.0).all()
    wn = dec(w) if weight else np.ones(cols)
    yn, mn, rn = dec(dy), dec(mean), dec(rstd)
    rx, rw, rb = b128.layernorm_bwd(yn, hn, wn, mn, rn, dec(dh) if with_dh else None)
    # n is good to 3 roundings, the two sums to N of the sums of the sizes
    n = (hn - mn[:, None]) * rn[:, None]
    dn = 2.0 ** -22 * (np.abs(n) + np.abs(hn) * rn[:, None])
    g = yn * wn
    ka, kb = np.abs(g).mean(1, keepdims=True), np.abs(g * n).mean(1, keepdims=True)
    kn = (np.abs(g) * dn).mean(1, keepdims=True)
    tol = rn[:, None] * ((N + 2.0 ** -22) * ka + np.abs(n) * ((N + 2.0 ** -22) * kb + kn) + dn * kb +
                         2.0 ** -22 * (np.abs(g) + np.abs(n) * kb)) + 2.0 ** -23 * np.abs(rx)
    if with_dh:
        tol = tol + 2.0 ** -23 * np.abs(dec(dh))
    _near(dx[:, offset:], rx, tol, "dx")
    # a column's sum: at most ceil(rows / blocks) and 32 + 5 steps more
    steps = (rows / 100 + 64) * 2.0 ** -24
    if dw is not None:
        _near(dw, rw, (np.abs(yn) * (steps * np.abs(n) + dn)).sum(0), "dw")
    if db is not None:
        _near(db, rb, steps * np.abs(yn).sum(0), "db")
    return dx, dw, db


@pytest.mark.parametrize("rows,cols", SHAPES + [(257, 1536), (5000, 100), (40, 5120), (30, 12288)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("offset", [0, 3])
def test_backward(rows, cols, dtype, with_dh, offset):
    _backward(rows, cols, dtype, offset, with_dh)


@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 7), (5, 255), (7, 257), (300, 513), (160, 4096), (2, 8192), (30, 12288),
                                       (3, 16383), (2, 16384), (3, 16385)])
@pytest.mark.parametrize("fmt", [torch.float8_e4m3fn, torch.float8_e5m2])
@pytest.mark.parametrize("offset", [0, 3])
def test_backward_from_eight_bits(rows, cols, fmt, offset):
    _backward(rows, cols, TYPES[cols % 3], offset, True, fmt)


def test_backward_optional_parts():
    for kw in (dict(weight=False), dict(config=(True, False)), dict(config=(False, True)), dict(config=(False, False)),
               dict(h8=torch.float8_e4m3fn, config=(False, False), weight=False)):
        for cols in (300, 16400):
            _backward(40, cols, torch.bfloat16, 0, True, **kw)


def test_backward_repeats_bit_for_bit_and_in_place():
    a = _backward(900, 1536, torch.bfloat16, 0, True)
    b = _backward(900, 1536, torch.bfloat16, 0, True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    dy, h = _rand(300, 513, torch.bfloat16, 1), _rand(300, 513, torch.bfloat16, 2)
    mean, rstd = h.float().mean(1), h.float().var(1).rsqrt()
    for over in ("dy", "h", "dh"):
        t = {"dy": dy.clone(), "h": h.clone(), "dh": dy.clone()}
        want = torch.empty_like(dy)
        args = (t["dy"], t["h"], None, mean, rstd)
        gge.gge_layernorm_bwd(*args, want, dH=t["dh"])
        gge.gge_layernorm_bwd(*args, t[over], dH=t["dh"])
        assert torch.equal(t[over], want)


def test_no_rows_and_scale_orders():
    dw, db = torch.full((70,), 5.0, device=DEV), torch.full((70,), 5.0, device=DEV)
    e = torch.empty(0, 70, dtype=torch.bfloat16, device=DEV)
    gge.gge_layernorm_bwd(e, e, None, torch.empty(0, device=DEV), torch.empty(0, device=DEV), torch.empty_like(e), dW=dw, dB=db)
    assert not dw.any() and not db.any()
    gge.gge_layernorm(e, Y=torch.empty_like(e), Q=gge.b128_empty(0, 70, device=DEV))
    # scales row by row
    x = _rand(30, 300, torch.bfloat16, 1)
    q = gge.B128Tensor(_empty(30, 300).codes, torch.empty(30, 3, device=DEV))
    q2 = _empty(30, 300)
    gge.gge_layernorm(x, Q=q, H8=q2)
    q3, h3 = _empty(30, 300), gge.B128Tensor(_empty(30, 300).codes, torch.empty(30, 3, device=DEV))
    gge.gge_layernorm(x, Q=q3, H8=h3)
    assert torch.equal(q.scales, q3.scales) and np.array_equal(_numbers(q), _numbers(q3))
    assert torch.equal(q2.scales, h3.scales)


def test_captured_beside_an_eager_call():
    """A captured forward and backward replay with new data; the partial sums are the graph's own."""
    x, w = _rand(200, 1000, torch.bfloat16, 1), _rand(1, 1000, torch.bfloat16, 2)[0]
    dy = _rand(200, 1000, torch.bfloat16, 3)

    def step():
        mean, rstd, h8 = torch.empty(200, device=DEV), torch.empty(200, device=DEV), gge.b128_empty(200, 1000, device=DEV)
        dx, dw, db = torch.empty_like(x), torch.empty(1000, device=DEV), torch.empty(1000, device=DEV)
        gge.gge_layernorm(x, w, H8=h8, mean=mean, rstd=rstd)
        gge.gge_layernorm_bwd(dy, h8, w, mean, rstd, dx, dW=dw, dB=db)
        return dx, dw, db

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    graph.replay()
    eager = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, eager))
    x.mul_(2).add_(1)
    graph.replay()
    eager2 = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, eager2)) and not torch.equal(eager[0], eager2[0])


def test_arguments_refused():
    x = _rand(10, 256, torch.bfloat16, 1)
    m = torch.empty(10, device=DEV)
    with pytest.raises(ValueError):
        gge.gge_layernorm(x, torch.ones(255, device=DEV))
    with pytest.raises(TypeError):
        gge.gge_layernorm(x, torch.ones(256, device=DEV), torch.ones(256, device=DEV).half())
    with pytest.raises(gge.GgeError):
        gge.gge_layernorm(x, Y=torch.empty(10, 256, device=DEV))
    with pytest.raises(gge.GgeError):
        gge.gge_layernorm(x, residual_out=x)
    with pytest.raises(gge.GgeError):
        gge.gge_layernorm(x, Q=gge.b128_empty(10, 256, 128, device=DEV))
    with pytest.raises(gge.GgeError):
        gge.gge_layernorm_bwd(x, None, None, m, m, torch.empty_like(x))
    with pytest.raises(gge.GgeError):
        gge.gge_layernorm_bwd(x, gge.b128_empty(10, 128, device=DEV), None, m, m, torch.empty_like(x))
    with pytest.raises(gge.GgeError):
        gge.gge_layernorm_bwd(x, x, None, m, m, torch.empty_like(x), dW=torch.empty(256, device=DEV),
                              workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
