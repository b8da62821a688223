"""RMS norm with the residual's addition, its quantised outputs and its backward, on
the GPU against the float64 oracle.

Tolerances.  A row's sum of squares is added up in fp32 in at most 64 steps one after
the other, so it is off by at most 64 * 2^-24 relatively, inv by half of that and
rsqrt's 2^-22; y's two products add 2^-23: REL below covers them.  Outputs are rounded
once more: one spacing of their type.  The backward's sums cancel, so their bounds are
relative to the sums of the sizes."""

import numpy as np
import pytest
import torch

from grouped_gemm_epilogues_gb300 import binding as gge
from oracle import formats, lowp

from helpers import FMT, dec

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
EPS = 1e-5
REL = 64 * 2.0 ** -24 + 2.0 ** -21
TYPES = (torch.bfloat16, torch.float16, torch.float32)


def _rand(rows, cols, dtype, seed, offset=0):
    """A (rows, cols) device matrix; `offset` elements into wider rows (any alignment)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols + offset, generator=g) * torch.exp(0.5 * torch.randn(cols + offset, generator=g))
    return x.to(dtype).to(DEV)[:, offset:]


def _near(got, ref, rel, what):
    fmt = FMT[got.dtype]
    got = dec(got)
    tol = rel * np.abs(ref) + formats.quantum(ref, fmt)
    assert np.isfinite(got).all(), what
    worst = np.max(np.abs(got - ref) / tol) if got.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the tolerance"


SHAPES = [(1, 1), (1, 8), (2, 7), (3, 64), (5, 255), (4, 256), (7, 257), (300, 513), (9, 2049), (160, 4096),
          (2, 8192), (700, 1000), (3, 16383), (2, 16384), (3, 16385), (2, 40001)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("offset", [0, 3])
def test_forward(rows, cols, dtype, residual, offset):
    x, w = _rand(rows, cols, dtype, 1, offset), _rand(1, cols, dtype, 2)[0]
    r = _rand(rows, cols, dtype, 3, offset) if residual else None
    y = torch.full((rows, cols + offset), 9.0, dtype=dtype, device=DEV)
    h = torch.full((rows, cols + offset), 9.0, dtype=dtype, device=DEV) if residual else None
    inv = torch.empty(rows, device=DEV)
    gge.gge_rmsnorm(x, w, Y=y[:, offset:], residual=r, residual_out=h[:, offset:] if residual else None,
                    inv_rms=inv, eps=EPS)
    rh, rinv, ry = lowp.rmsnorm(dec(x), dec(w), EPS, dec(r) if residual else None, FMT[dtype])
    assert (y[:, :offset] == 9.0).all()
    if residual:
        assert np.array_equal(dec(h[:, offset:]), rh)
        assert (h[:, :offset] == 9.0).all()
    _near(inv, rinv, REL, "inv")
    _near(y[:, offset:], ry, REL, "y")


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 64), (5, 255), (7, 300), (300, 513), (160, 4096), (9, 2056),
                                       (2, 16384), (3, 16385)])
@pytest.mark.parametrize("offset", [0, 1])
def test_quantised_output(fmt, rows, cols, offset):
    """Scales fit the unrounded y's blocks, and every value is within half a spacing of its
    code's grid of it (both up to the fp32 error of y)."""
    dtype = TYPES[cols % 2]
    x, r, w = _rand(rows, cols, dtype, 4, offset), _rand(rows, cols, dtype, 5, offset), _rand(1, cols, torch.float32, 6)[0]
    _, _, ry = lowp.rmsnorm(dec(x), dec(w), EPS, dec(r), FMT[dtype])
    t = torch.tensor([np.abs(ry).max() / 2688], dtype=torch.float32, device=DEV) if fmt == "nvfp4" else None
    tv = float(t.cpu()) if t is not None else 1.0
    q = gge.mx_empty(rows, cols, fmt, device=DEV, tensor_scale=t)
    q.codes.fill_(0xA5)
    q.scales.fill_(0xA5)
    h = torch.empty(rows, cols, dtype=dtype, device=DEV)
    vals = torch.full((rows, cols + offset), 9.0, dtype=torch.float32, device=DEV)
    gge.gge_rmsnorm(x, w, residual=r, residual_out=h, Q=q, values=vals[:, offset:], eps=EPS)
    codes, flat = q.codes.cpu().numpy(), q.scales.cpu().numpy()
    got = lowp.decode(codes, flat, rows, cols, fmt, tv)
    assert np.array_equal(dec(vals[:, offset:]), formats.round_to(got, formats.F32))
    assert (vals[:, :offset] == 9.0).all()
    byte, padding = lowp.scale_bytes(flat, rows, cols, fmt)
    assert not padding.any()
    per = 8 if fmt == "mxfp8" else 4
    assert not np.unpackbits(codes, axis=1, bitorder="little")[:, cols * per:].any()
    size = lowp.BLOCK[fmt]
    nb = byte.shape[1]
    pad = np.zeros((rows, nb * size))
    pad[:, :cols] = ry
    amax = np.abs(pad.reshape(rows, nb, size)).max(2)
    if fmt == "nvfp4":
        s = formats.decode(byte, formats.E4M3)
        want = np.clip(amax / (6 * tv), 2.0 ** -9, 448.0)
        assert (np.abs(s - want) <= formats.quantum(want, formats.E4M3) / 2 + 2 * REL * want).all()
        unit = np.repeat(s * tv, size, 1)[:, :cols]
    else:
        s = np.ldexp(1.0, byte.astype(np.int64) - 127)
        top = lowp.TOP[fmt]
        assert (amax * (1 - 2 * REL) <= s * top).all()
        assert (amax * (1 + 2 * REL) > s * top / 2)[byte > 0].all()
        unit = np.repeat(s, size, 1)[:, :cols]
    scaled = np.abs(ry) / unit
    if fmt == "mxfp8":
        half = formats.quantum(np.minimum(scaled, 448.0), formats.E4M3) / 2
    else:
        half = np.where(scaled < 2, 0.25, np.where(scaled < 4, 0.5, 1.0))
    # (nvfp4's scale may round down: what exceeds 6 of it saturates)
    limit = np.where(scaled > lowp.TOP[fmt], scaled - lowp.TOP[fmt], half)
    assert (np.abs(got - ry) <= unit * limit + 2 * REL * np.abs(ry)).all()


def test_norm_quantise_is_quantise_of_the_norm():
    """The fused output equals gge_mx_quantize of the fp32 y."""
    x, w = _rand(40, 1000, torch.float32, 7), _rand(1, 1000, torch.float32, 8)[0]
    y = torch.empty_like(x)
    q = gge.mx_empty(40, 1000, "mxfp4", device=DEV)
    gge.gge_rmsnorm(x, w, Y=y, Q=q, eps=EPS)
    q2 = gge.mx_empty(40, 1000, "mxfp4", device=DEV)
    gge.gge_mx_quantize(y, q2)
    assert torch.equal(q.codes, q2.codes)
    assert np.array_equal(*(lowp.scale_bytes(z.scales.cpu().numpy(), 40, 1000, "mxfp4")[0] for z in (q, q2)))


def test_forward_in_place_and_not_finite():
    """residual_out over the residual; an infinite value and a NaN stay in their rows."""
    x, r, w = _rand(50, 777, torch.bfloat16, 9), _rand(50, 777, torch.bfloat16, 10), _rand(1, 777, torch.bfloat16, 11)[0]
    x[7, 5], x[8, 6] = float("inf"), float("nan")
    rx, rr = dec(x), dec(r)
    y = torch.empty(50, 777, dtype=torch.bfloat16, device=DEV)
    gge.gge_rmsnorm(x, w, Y=y, residual=r, residual_out=r, eps=EPS)
    ok = np.setdiff1d(np.arange(50), [7, 8])
    h, _, ry = lowp.rmsnorm(rx[ok], dec(w), EPS, rr[ok], formats.BF16)
    assert np.array_equal(dec(r)[ok], h)
    _near(y[torch.from_numpy(ok).to(DEV)], ry, REL, "y")
    assert torch.isnan(y[8].float()).all() and torch.isnan(y[7, 5].float())


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("offset", [0, 5])
def test_backward(rows, cols, dtype, with_dh, offset):
    dy, h = _rand(rows, cols, dtype, 12, offset), _rand(rows, cols, dtype, 13, offset)
    w = _rand(1, cols, torch.float32 if cols % 2 else dtype, 14)[0]
    dh = _rand(rows, cols, dtype, 15, offset) if with_dh else None
    inv = torch.rsqrt(h.float().square().mean(1) + EPS)
    dx = torch.full((rows, cols + offset), 9.0, dtype=dtype, device=DEV)
    dw = torch.full((cols,), float("nan"), device=DEV)
    gge.gge_rmsnorm_bwd(dy, h, w, inv, dx[:, offset:], dW=dw, dH=dh)
    a, b, wv, iv = dec(dy), dec(h), dec(w), dec(inv)
    rdx, rdw = lowp.rmsnorm_bwd(a, b, wv, iv, dec(dh) if with_dh else None)
    assert (dx[:, :offset] == 9.0).all()
    # the sizes that cancel: each term of dx, and of the dot product under it
    i = iv[:, None]
    size = np.abs(i * a * wv) + np.abs(i * b) * i * i * (np.abs(a * wv) * np.abs(b)).mean(1, keepdims=True)
    size = size + (np.abs(dec(dh)) if with_dh else 0.0)
    tol = REL * size + formats.quantum(rdx, FMT[dtype])
    assert (np.abs(dec(dx[:, offset:]) - rdx) <= tol).all()
    # dw: sums over the rows, in fp32 along a block's rows and then over the blocks
    steps = (rows + 151) // 152 + 152 + 32
    tol = (steps * 2.0 ** -24 + 2.0 ** -22) * np.abs(a * b * i).sum(0) + formats.quantum(rdw, formats.F32)
    assert (np.abs(dec(dw) - rdw) <= tol).all()
    dw2 = torch.empty_like(dw)
    gge.gge_rmsnorm_bwd(dy, h, w, inv, dx[:, offset:], dW=dw2, dH=dh)
    assert torch.equal(dw, dw2), "the order of dw's sum is fixed"


@pytest.mark.parametrize("cols", [1000, 1003, 20000])
def test_backward_in_place_without_dw_and_no_rows(cols):
    dy, h, w = _rand(30, cols, torch.bfloat16, 16), _rand(30, cols, torch.bfloat16, 17), _rand(1, cols, torch.bfloat16, 18)[0]
    inv = torch.rsqrt(h.float().square().mean(1) + EPS)
    dx, dw = torch.empty_like(dy), torch.empty(cols, device=DEV)
    gge.gge_rmsnorm_bwd(dy, h, w, inv, dx, dW=dw, dH=h)
    only = torch.empty_like(dy)
    gge.gge_rmsnorm_bwd(dy, h, w, inv, only, dH=h)
    assert torch.equal(only, dx)
    dw2 = torch.empty_like(dw)
    gge.gge_rmsnorm_bwd(dy, h, w, inv, h, dW=dw2, dH=h)          # over h and dh
    assert torch.equal(h, dx) and torch.equal(dw, dw2)
    gge.gge_rmsnorm_bwd(dy[:0], dy[:0], w, inv[:0], dy[:0], dW=dw2)
    assert not dw2.any()


def test_backward_against_differences_of_the_forward():
    """The gradient of a scalar of the GPU's own forward (fp32), by central differences."""
    rows, cols = 4, 64
    x, w = _rand(rows, cols, torch.float32, 19), _rand(1, cols, torch.float32, 20)[0]
    g = _rand(rows, cols, torch.float32, 21)

    def forward(x, w):
        y, inv = torch.empty_like(x), torch.empty(rows, device=DEV)
        gge.gge_rmsnorm(x, w, Y=y, inv_rms=inv, eps=EPS)
        return (y.double() * g.double()).sum().item(), inv

    _, inv = forward(x, w)
    dx, dw = torch.empty_like(x), torch.empty(cols, device=DEV)
    gge.gge_rmsnorm_bwd(g, x, w, inv, dx, dW=dw)
    d = 2.0 ** -6
    # the forward's outputs are off by about 2^-23 of their size each; divided by 2 d
    noise = 2.0 ** -22 * float(g.abs().sum()) * float(w.abs().max()) * 4 / (2 * d)
    for i, j in [(0, 0), (1, 13), (3, 63)]:
        e = torch.zeros_like(x)
        e[i, j] = d
        diff = (forward(x + e, w)[0] - forward(x - e, w)[0]) / (2 * d)
        # third-order term of the difference: below d^2 times a few of the row's gradients
        assert abs(diff - dx[i, j].item()) <= noise + 10 * d * d * (1 + float(dx[i].abs().max()))
    for j in (0, 31):
        e = torch.zeros_like(w)
        e[j] = d
        diff = (forward(x, w + e)[0] - forward(x, w - e)[0]) / (2 * d)
        assert abs(diff - dw[j].item()) <= noise


def test_norm_streams_and_graph():
    x, w = _rand(64, 1000, torch.bfloat16, 22), _rand(1, 1000, torch.bfloat16, 23)[0]
    outs = [torch.empty_like(x) for _ in range(3)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        gge.gge_rmsnorm(x, w, Y=outs[0], eps=EPS)
    gge.gge_rmsnorm(x, w, Y=outs[1], eps=EPS)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gge.gge_rmsnorm(x, w, Y=outs[2], eps=EPS)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[1], outs[2])


# Rows a row group takes one after the other, on no particular boundary: starting at
# the same place in every tensor (one offset), or not (several).
MANY = [(9999, 77), (5000, 1003), (1300, 4099), (700, 8185)]
OFFSETS = [(0, 0, 0, 0), (5, 5, 5, 5), (1, 3, 0, 6)]


@pytest.mark.parametrize("rows,cols", MANY)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offsets", OFFSETS)
def test_forward_many_rows(rows, cols, dtype, offsets):
    x, r = (_rand(rows, cols, dtype, 21 + i, offsets[i]) for i in (0, 1))
    w = _rand(1, cols, dtype, 25)[0]
    h, y = (torch.full((rows, cols + o + 16), 9.0, dtype=dtype, device=DEV) for o in offsets[2:])
    hv, yv = h[:, offsets[2]:][:, :cols], y[:, offsets[3]:][:, :cols]
    inv = torch.empty(rows, device=DEV)
    gge.gge_rmsnorm(x, w, Y=yv, residual=r, residual_out=hv, inv_rms=inv, eps=EPS)
    rh, rinv, ry = lowp.rmsnorm(dec(x), dec(w), EPS, dec(r), FMT[dtype])
    assert np.array_equal(dec(hv), rh)
    _near(inv, rinv, REL, "inv")
    _near(yv, ry, REL, "y")
    for t, o in ((h, offsets[2]), (y, offsets[3])):
        assert (t[:, :o] == 9.0).all() and (t[:, cols + o:] == 9.0).all()


@pytest.mark.parametrize("rows,cols", MANY)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_forward_many_rows_alone(rows, cols, dtype, pad):
    """x to y without a residual; y's rows `pad` elements wider than x's."""
    x, w = _rand(rows, cols, dtype, 31), _rand(1, cols, torch.float32, 32)[0]
    y = torch.full((rows, cols + pad), 9.0, dtype=dtype, device=DEV)
    gge.gge_rmsnorm(x, w, Y=y[:, :cols], eps=EPS)
    _, _, ry = lowp.rmsnorm(dec(x), dec(w), EPS, None, FMT[dtype])
    _near(y[:, :cols], ry, REL, "y")
    assert (y[:, cols:] == 9.0).all()


@pytest.mark.parametrize("cols", [77, 1000, 1003])
@pytest.mark.parametrize("offset", [0, 3])
def test_one_residual_row_for_all(cols, offset):
    x, w = _rand(3000, cols, torch.bfloat16, 41, offset), _rand(1, cols, torch.bfloat16, 42)[0]
    r = _rand(1, cols, torch.bfloat16, 43, offset).expand(3000, cols)
    h, y = torch.empty(3000, cols, dtype=torch.bfloat16, device=DEV), torch.empty_like(x)
    gge.gge_rmsnorm(x, w, Y=y, residual=r, residual_out=h, eps=EPS)
    rh, _, ry = lowp.rmsnorm(dec(x), dec(w), EPS, dec(r), FMT[torch.bfloat16])
    assert np.array_equal(dec(h), rh)
    _near(y, ry, REL, "y")


@pytest.mark.parametrize("rows,cols", MANY + [(400, 8193), (400, 12001)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offsets", OFFSETS)
def test_backward_many_rows(rows, cols, dtype, offsets):
    dy, h, dh = (_rand(rows, cols, dtype, 51 + i, offsets[i]) for i in range(3))
    w = _rand(1, cols, dtype, 55)[0]
    inv = torch.rsqrt(h.float().square().mean(1) + EPS)
    dx = torch.full((rows, cols + offsets[3]), 9.0, dtype=dtype, device=DEV)
    dw = torch.full((cols,), float("nan"), device=DEV)
    gge.gge_rmsnorm_bwd(dy, h, w, inv, dx[:, offsets[3]:], dW=dw, dH=dh)
    a, b, wv, iv = dec(dy), dec(h), dec(w), dec(inv)
    rdx, rdw = lowp.rmsnorm_bwd(a, b, wv, iv, dec(dh))
    assert (dx[:, :offsets[3]] == 9.0).all()
    i = iv[:, None]
    size = np.abs(i * a * wv) + np.abs(i * b) * i * i * (np.abs(a * wv) * np.abs(b)).mean(1, keepdims=True) + np.abs(dec(dh))
    assert (np.abs(dec(dx[:, offsets[3]:]) - rdx) <= REL * size + formats.quantum(rdx, FMT[dtype])).all()
    steps = (rows + 151) // 152 + 152 + 32
    tol = (steps * 2.0 ** -24 + 2.0 ** -22) * np.abs(a * b * i).sum(0) + formats.quantum(rdw, formats.F32)
    assert (np.abs(dec(dw) - rdw) <= tol).all()


@pytest.mark.parametrize("cols", [1000, 1003])
def test_captured_backward_then_a_wider_call(cols):
    """A graph's dW has to stay right, and other tensors untouched, after a wider call and new
    allocations between the capture and the replay."""
    dy, h = (_rand(300, cols, torch.bfloat16, s) for s in (61, 62))
    w = _rand(1, cols, torch.bfloat16, 63)[0]
    inv = torch.rsqrt(h.float().square().mean(1) + EPS)
    dx, dw = torch.empty_like(dy), torch.empty(cols, device=DEV)
    gge.gge_rmsnorm_bwd(dy, h, w, inv, dx, dW=dw)
    want_dx, want_dw = dx.clone(), dw.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gge.gge_rmsnorm_bwd(dy, h, w, inv, dx, dW=dw)
    wide = [_rand(300, 12000, torch.bfloat16, s) for s in (64, 65)]
    wdx, wdw = torch.empty_like(wide[0]), torch.empty(12000, device=DEV)
    winv = torch.rsqrt(wide[1].float().square().mean(1) + EPS)
    gge.gge_rmsnorm_bwd(wide[0], wide[1], _rand(1, 12000, torch.bfloat16, 66)[0], winv, wdx, dW=wdw)
    others = [torch.full((n,), 7.0, device=DEV) for n in (1 << 18, 1 << 20, 1 << 22) for _ in range(8)]
    dx.fill_(9.0)
    dw.fill_(9.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx, want_dx) and torch.equal(dw, want_dw)
    assert all((t == 7.0).all() for t in others)


def test_backward_on_two_streams_at_once():
    """Calls without a workspace of the caller's do not share their partial sums."""
    cases = []
    for i, cols in enumerate((1536, 2000)):
        dy, h = (_rand(4000, cols, torch.bfloat16, 71 + 2 * i + j) for j in (0, 1))
        w, inv = _rand(1, cols, torch.bfloat16, 75 + i)[0], torch.rsqrt(h.float().square().mean(1) + EPS)
        want = torch.empty(cols, device=DEV)
        gge.gge_rmsnorm_bwd(dy, h, w, inv, torch.empty_like(dy), dW=want)
        cases.append((torch.cuda.Stream(), (dy, h, w, inv, torch.empty_like(dy)), want,
                      [torch.empty_like(want) for _ in range(10)]))
    torch.cuda.synchronize()
    for n in range(10):
        for stream, args, _, dws in cases:
            with torch.cuda.stream(stream):
                gge.gge_rmsnorm_bwd(*args, dW=dws[n])
    torch.cuda.synchronize()
    for _, _, want, dws in cases:
        assert all(torch.equal(want, d) for d in dws)
