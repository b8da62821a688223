"""8-bit matrices with a scale for each block of 128 on the GPU against the float64 oracle:
quantisation, transposition, and the product with its epilogues.

Quantisation is exact (its fp32 operations are the definition): codes and scales have to be
equal.  Products are compared within 1e-5 * sum |a b| + 1 ulp of the output, the bound of the
other products: a block's sum on the tensor core is good to a few 2^-24, its scale's product and
the addition to the sum round once each, so k blocks are off by (k + 3) 2^-24 of sum |a b| at
most, 8e-6 for the 128 blocks of the longest K here.  gelu_tanh and silu add 2^-20 of the value
they are taken of (the SFU's exponential and reciprocal, 2^-22 each), act' 1e-6 of |S|'s terms.
An 8-bit output is off by half a step of its code's grid beside that."""

import numpy as np
import pytest
import torch

from grouped_gemm_epilogues_gb300 import binding as gge
from oracle import activations, b128, formats, gemm as og

from helpers import FMT, check, dec

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
CODES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
NAME = {v: k for k, v in CODES.items()}


def _x(rows, cols, dtype=torch.bfloat16, seed=0, spread=1.0):
    """Values whose rows differ in size, with zeros and a row of them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(spread * torch.randn(rows, 1, generator=g).clamp(-2, 2))
    x[torch.rand(rows, cols, generator=g) < 0.05] = 0.0
    if rows > 2:
        x[1] = 0.0
    return x.to(dtype)


def _empty(rows, cols, block_rows=1, fmt="e4m3", batch=None):
    q = gge.b128_empty(rows, cols, block_rows, CODES[fmt], DEV, batch)
    q.codes.view(torch.uint8).fill_(0xA5)
    q.scales.fill_(float("nan"))
    return q


def _parts(q):
    return q.codes.contiguous().view(torch.uint8).cpu().numpy(), q.scales.cpu().numpy()


def _numbers(q):
    codes, scales = _parts(q)
    f = NAME[q.dtype]
    if codes.ndim == 2:
        return b128.decode(codes, scales, f, q.block_rows)
    return np.stack([b128.decode(c, s, f, q.block_rows) for c, s in zip(codes, scales)])


def _check_codes(x, q):
    ref, scale = b128.quantise(x, NAME[q.dtype], q.block_rows)
    got = _numbers(q)
    assert np.array_equal(q.scales.cpu().numpy().astype(np.float64), scale, equal_nan=True)
    assert np.array_equal(got, ref, equal_nan=True)
    return ref


def _held(x, block_rows=1, fmt="e4m3"):
    """A CPU matrix (or batch) quantised on the GPU, and its numbers."""
    q = _empty(x.shape[-2], x.shape[-1], block_rows, fmt, x.shape[0] if x.dim() == 3 else None)
    gge.gge_b128_quantize(x.to(DEV), q)
    return q, _numbers(q)


SHAPES = [(1, 1), (1, 128), (3, 127), (7, 129), (130, 64), (64, 257), (129, 129), (5, 1000), (257, 2049)]


@pytest.mark.parametrize("fmt", CODES)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantise_is_exact(fmt, block_rows, transposed, rows, cols):
    dtype = (torch.bfloat16, torch.float16, torch.float32)[(rows + cols) % 3]
    x = _x(rows, cols, dtype, seed=rows, spread=3.0)
    src = x.t().contiguous().to(DEV).t() if transposed else x.to(DEV)
    q = _empty(rows, cols, block_rows, fmt)
    v = torch.full((rows, cols), 7.0, dtype=torch.float32, device=DEV)
    gge.gge_b128_quantize(src, q, values=v)
    ref = _check_codes(dec(x), q)
    assert np.array_equal(dec(v), formats.round_to(ref, formats.F32))


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("values", [torch.bfloat16, torch.float16, torch.float32])
def test_quantise_values_types_and_round_trip(block_rows, transposed, values):
    x = _x(140, 301, torch.bfloat16, seed=4, spread=0.5)
    src = x.t().contiguous().to(DEV).t() if transposed else x.to(DEV)
    q = _empty(140, 301, block_rows)
    v = torch.empty(140, 304, dtype=values, device=DEV)
    for at in (v[:, :301], v[:, 3:304]):      # rows on 16 bytes, and elsewhere
        v.fill_(7.0)
        gge.gge_b128_quantize(src, q, values=at)
        ref = _check_codes(dec(x), q)
        # (the number is an fp32 product, rounded once more to 16 bits)
        want = formats.round_to(formats.round_to(ref, formats.F32), FMT[values])
        assert np.array_equal(dec(at), want)
        at.fill_(7.0)
        assert (v == 7.0).all()
        gge.gge_b128_dequantize(q, at)
        assert np.array_equal(dec(at), want)


@pytest.mark.parametrize("fmt", CODES)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("transposed", [False, True])
def test_quantise_extremes_and_not_finite(fmt, block_rows, transposed):
    x = torch.zeros(260, 300)
    x[0, :32] = 3.0e38
    x[1, 130:140] = 2.0 ** -140
    x[2, 0], x[3, 299] = float("inf"), float("nan")
    x[150, 200] = float("-inf")
    x[200, :100] = torch.linspace(-1, 1, 100)
    x[259] = 448.0
    src = x.t().contiguous().to(DEV).t() if transposed else x.to(DEV)
    q = _empty(260, 300, block_rows, fmt)
    gge.gge_b128_quantize(src, q)
    _check_codes(dec(x), q)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("transposed", [False, True])
def test_quantise_strided_batches_scale_orders_and_guards(block_rows, transposed):
    """Rows that start on odd elements, batches, scales row by row, and what lies beside."""
    g = torch.Generator().manual_seed(2)
    big = torch.randn(3, 160, 211, generator=g).bfloat16().to(DEV)
    x = big[:, 1:151, 3:202].transpose(1, 2) if transposed else big[:, 1:151, 3:202]
    rows, cols = x.shape[1:]
    codes = torch.full((3, rows + 1, cols // 16 * 16 + 48), 0x5A, dtype=torch.uint8, device=DEV)
    scales = torch.full((3, 2, 200, 3), 5.0, device=DEV)
    at = scales[:, 0, :-(-rows // block_rows), :2]
    q = gge.B128Tensor(codes[:, :rows, :cols].view(torch.float8_e4m3fn), at, block_rows)
    gge.gge_b128_quantize(x, q)
    for b in range(3):
        one = gge.B128Tensor(q.codes[b], q.scales[b], block_rows)
        _check_codes(dec(x[b]), one)
    codes[:, :rows, :cols] = 0x5A
    at.fill_(5.0)
    assert (codes == 0x5A).all() and (scales == 5.0).all()


@pytest.mark.parametrize("fmt", CODES)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("from_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 127), (7, 129), (130, 64), (200, 257), (257, 1030)])
def test_transpose_is_exact(fmt, block_rows, from_rows, rows, cols):
    other = "e5m2" if fmt == "e4m3" and cols % 2 else "e4m3"
    x, _ = _held(_x(rows, cols, seed=cols), from_rows, other)
    q = _empty(cols, rows, block_rows, fmt)
    v = torch.full((cols, rows), 7.0, dtype=torch.bfloat16, device=DEV)
    gge.gge_b128_transpose(x, q, values=v)
    # (its numbers are fp32 products of code and scale)
    turned = formats.round_to(_numbers(x), formats.F32).T
    ref = _check_codes(turned, q)
    assert np.array_equal(dec(v), formats.round_to(formats.round_to(ref, formats.F32), formats.BF16))


def test_transpose_batches_and_not_finite():
    x = torch.stack([_x(70, 140, torch.float32, 3), _x(70, 140, torch.float32, 4)])
    x[1, 5, 130] = float("nan")
    q, _ = _held(x)
    t = _empty(140, 70, 1, "e4m3", 2)
    gge.gge_b128_transpose(q, t)
    for b in range(2):
        with np.errstate(invalid="ignore"):
            turned = formats.round_to(_numbers(q)[b], formats.F32).T
        _check_codes(turned, gge.B128Tensor(t.codes[b], t.scales[b]))


# ---------------------------------------------------------------- products

def _status():
    torch.cuda.synchronize()
    return gge.gge_read_device_status()[0]


def _check_q(q, want, tol):
    """8-bit outputs: codes round from within tol of `want`, scales fit."""
    got = _numbers(q)
    scales = q.scales.cpu().numpy()
    assert np.isfinite(got).all()
    value, scale = b128.off_codes(got, scales, want, tol, NAME[q.dtype])
    assert value <= 1.0 and scale <= 1.0, (value, scale)


def _slack(act, v, bound):
    """Tolerance of act(v) for a v that is off by 1e-5 * bound, beside the SFU's."""
    lip = activations.lipschitz(act, v)
    if act == "relu_sq":      # (its slope 2 v is not that of v + 1e-5 bound)
        return 1e-5 * lip * bound + (1e-5 * bound) ** 2
    return 1e-5 * lip * bound + (np.abs(v) * 2.0 ** -20 if act in ("gelu_tanh", "silu") else 0.0)


def _product(m, n, k, b_rows=128, a_rows=1, act="none", c=None, d=torch.bfloat16, p=torch.bfloat16, alpha=1.0,
             beta=0.0, batch=None, config=None, dev_scalars=False, seed=0, fmts=("e4m3", "e4m3"), spread=0.7):
    """d, p and c: None, a value type, or the name of an 8-bit one."""
    lead = (batch,) if batch else ()
    mats = []
    for rows, s, block, f in ((m, seed, a_rows, fmts[0]), (n, seed + 1, b_rows, fmts[1])):
        x = torch.stack([_x(rows, k, seed=s + 10 * b, spread=spread) for b in range(batch or 1)])
        mats.append(_held(x if batch else x[0], block, f))
    (A, av), (B, bv) = mats
    g = torch.Generator().manual_seed(seed + 99)
    C = cv = None
    if c is not None:
        C = torch.randn(*lead, m, n, generator=g)
        if isinstance(c, str):
            C, cv = _held(C, 1, c)
        else:
            C = C.to(c)
            cv = dec(C)
            C = C.to(DEV)

    def room(t):
        if t is None:
            return None
        if isinstance(t, str):
            return _empty(m, n, 1, t, batch)
        return torch.full((*lead, m, n), float("nan"), dtype=t, device=DEV)

    D, P = room(d), room(p) if act != "none" else None
    kw = dict(alpha=alpha, beta=beta)
    if dev_scalars:
        kw = dict(alpha=99.0, beta=99.0, alpha_dev=torch.tensor([alpha], device=DEV),
                  beta_dev=torch.tensor([beta], device=DEV))
    gge.gge_gemm_b128(A, B, D=D, C=C, PostAct=P, act=act, config=config, **kw)
    assert _status() == "GGE_OK"
    as3 = (lambda v: v) if batch else (lambda v: v[None])
    ref = og.gemm(as3(av), as3(bv), None if cv is None else as3(cv), alpha=alpha, beta=beta, act=act)
    for out, t, name, want in ((D, d, "none", ref["v"]), (P, p, act, activations.apply(act, ref["v"]))):
        if out is None:
            continue
        tol = _slack(name, ref["v"], ref["bound"])
        if isinstance(t, str):
            for b in range(batch or 1):
                q = gge.B128Tensor(out.codes[b], out.scales[b]) if batch else out
                _check_q(q, want[b], tol[b])
        else:
            got, fmt = dec(out).reshape(want.shape), FMT[t]
            r = formats.round_to(want, fmt)
            fin = np.isfinite(r)     # (past its type's range an output is an infinity in both)
            assert np.array_equal(got[~fin], r[~fin])
            worst = np.max(np.abs(got[fin] - r[fin]) / (tol[fin] + formats.quantum(r[fin], fmt)))
            assert worst <= 1.0, (name, worst)
    return D, P


@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("m,n,k", [(1, 8, 1), (1, 264, 200), (2, 72, 31), (16, 512, 1024), (63, 136, 96),
                                   (64, 128, 33), (65, 128, 640), (127, 200, 257), (129, 264, 512),
                                   (300, 520, 1100), (257, 8, 2080)])
def test_product_shapes(b_rows, m, n, k):
    _product(m, n, k, b_rows, seed=m)


@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("tile_n", [256, 128, 64])
@pytest.mark.parametrize("m,n,k", [(300, 520, 1100), (70, 264, 4000), (600, 1032, 300)])
def test_every_tile_shape(b_rows, tile_n, m, n, k):
    """Each tile shape on the same problems, whole (one or several tiles a CTA) and, where the
    shape allows it, split along K over a cluster."""
    for kw in (dict(), dict(flags=32), dict(num_ctas=4), dict(flags=128, raster_band=2), dict(stages=2)):
        _product(m, n, k, b_rows, act="silu", config=gge.make_config(tile_n=tile_n, **kw), seed=tile_n)


@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("m,n,k", [(16, 128, 8192), (16, 1024, 8192), (40, 4096, 4096), (100, 256, 8192),
                                   (128, 2048, 2048), (128, 256, 16384)])
def test_split_k_clusters(b_rows, m, n, k):
    """Few tiles and a long K: the tile's sum comes from several CTAs.  Calls repeat bit for bit."""
    first = _product(m, n, k, b_rows, act="gelu_tanh", c=torch.bfloat16, beta=0.5, seed=3)
    again = _product(m, n, k, b_rows, act="gelu_tanh", c=torch.bfloat16, beta=0.5, seed=3)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("splits_k", [200, 4096])
@pytest.mark.parametrize("tile_n", [0, 256, 128])
def test_eight_bit_outputs(tile_n, splits_k):
    for m, n in ((130, 264), (33, 72), (257, 520)):
        cfg = gge.make_config(tile_n=tile_n)
        _product(m, n, splits_k, act="silu", d="e4m3", p="e4m3", config=cfg, seed=m)
        _product(m, n, splits_k, act="gelu_tanh", d="e5m2", p=torch.bfloat16, c=torch.float16, beta=0.5, config=cfg, seed=m)
        _product(m, n, splits_k, act="relu", d=None, p="e5m2", c="e4m3", beta=-1.0, alpha=0.5, config=cfg, seed=m)
        _product(m, n, splits_k, d="e4m3", config=cfg, seed=m)


@pytest.mark.parametrize("act", ["relu", "gelu_tanh", "silu", "relu_sq"])
@pytest.mark.parametrize("tile_n", [256, 128, 64])
def test_epilogues(act, tile_n):
    cfg = gge.make_config(tile_n=tile_n)
    _product(130, 264, 520, act=act, c=torch.float32, d=torch.float32, p=torch.float16, alpha=0.75, beta=-0.5, config=cfg)
    _product(130, 264, 520, 1, act=act, c=torch.float16, d=torch.float16, p=torch.float32, alpha=0.75, beta=0.5,
             config=cfg, dev_scalars=True)
    _product(130, 264, 520, act=act, d=None, config=cfg)
    _product(130, 264, 520, act=act, c="e4m3", beta=1.0, config=cfg)


@pytest.mark.parametrize("fmts", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("a_rows,b_rows", [(1, 1), (1, 128), (128, 1), (128, 128)])
def test_code_types_and_blocks(fmts, a_rows, b_rows):
    _product(300, 264, 700, b_rows, a_rows, fmts=fmts)


@pytest.mark.parametrize("tile_n", [0, 256, 128, 64])
@pytest.mark.parametrize("b_rows", [1, 128])
def test_batches(tile_n, b_rows):
    _product(70, 136, 300, b_rows, c=torch.bfloat16, beta=1.0, batch=3, config=gge.make_config(tile_n=tile_n))
    if tile_n != 64:
        _product(70, 136, 300, b_rows, act="silu", d="e4m3", p="e4m3", batch=3, config=gge.make_config(tile_n=tile_n))


def test_scales_in_any_order():
    """Scales row by row, or one for a whole matrix (stride 0), give the same product."""
    (A, _), (B, _) = _held(_x(100, 700)), _held(_x(72, 700, seed=5), 128)
    D = [torch.empty(100, 72, device=DEV) for _ in range(2)]
    gge.gge_gemm_b128(A, B, D=D[0])
    A2 = gge.B128Tensor(A.codes, A.scales.contiguous())
    B2 = gge.B128Tensor(B.codes, torch.stack((B.scales, B.scales), 2)[..., 1], 128)
    gge.gge_gemm_b128(A2, B2, D=D[1])
    assert torch.equal(*D)
    one = torch.full((1, 1), 0.25, device=DEV)
    gge.gge_gemm_b128(gge.B128Tensor(A.codes, one.expand(100, 6)), gge.B128Tensor(B.codes, one.expand(1, 6), 128), D=D[0])
    a, b = dec(A.codes), dec(B.codes)
    assert np.allclose(dec(D[0]), a @ b.T / 16, rtol=1e-5, atol=1e-5 * np.abs(a @ b.T).max())


def test_no_k_and_empty_sides():
    A, B = gge.b128_empty(40, 0, device=DEV), gge.b128_empty(64, 0, 128, device=DEV)
    C = torch.randn(40, 64, device=DEV).bfloat16()
    D = torch.full_like(C, float("nan"))
    gge.gge_gemm_b128(A, B, D=D, C=C, beta=0.5)
    assert torch.equal(D, (C.float() * 0.5).bfloat16())
    q = _empty(40, 64)
    gge.gge_gemm_b128(A, B, D=q, C=C, beta=1.0)
    _check_codes(dec(C), q)
    A = gge.b128_empty(0, 96, device=DEV)
    gge.gge_gemm_b128(A, gge.b128_empty(64, 96, device=DEV), D=torch.empty(0, 64, device=DEV))
    gge.gge_b128_quantize(torch.empty(0, 96, device=DEV), A)
    gge.gge_b128_transpose(A, gge.b128_empty(96, 0, device=DEV))
    assert _status() == "GGE_OK"


@pytest.mark.parametrize("tile_n", [256, 128, 64])
@pytest.mark.parametrize("b_rows", [1, 128])
def test_not_finite_rows_stay_in_their_rows(tile_n, b_rows):
    """A NaN block of A makes its row NaN and no other; a NaN value of B its row's (or its
    block's) columns.  An 8-bit output's block with a NaN is NaN throughout, and no other."""
    x, y = _x(70, 200, seed=5, spread=0.5), _x(264, 200, seed=6, spread=0.5)
    x[33, 100] = float("nan")
    y[140, 150] = float("inf")
    A, B = _held(x)[0], _held(y, b_rows)[0]
    D = torch.empty(70, 264, device=DEV)
    cfg = gge.make_config(tile_n=tile_n)
    gge.gge_gemm_b128(A, B, D=D, config=cfg)
    want = np.zeros((70, 264), dtype=bool)
    want[33] = True
    want[:, 128:256 if b_rows == 128 else 128] = True
    want[:, 140] = True
    assert np.array_equal(np.isnan(dec(D)), want)
    if tile_n != 64:
        q = _empty(70, 264)
        gge.gge_gemm_b128(A, B, D=q, config=cfg)
        bad = np.isnan(_numbers(q))
        assert bad[33].all() and bad[:, 128:256].all()
        rest = np.ones((70, 264), dtype=bool)
        rest[33], rest[:, 128:256] = False, False
        assert not bad[rest].any()


@pytest.mark.parametrize("tile_n", [256, 128, 64])
def test_output_guards_and_strides(tile_n):
    (A, av), (B, bv) = _held(_x(50, 160, seed=7)), _held(_x(72, 160, seed=8), 128)
    wide = torch.full((60, 96), 3.0, dtype=torch.bfloat16, device=DEV)
    cfg = gge.make_config(tile_n=tile_n)
    gge.gge_gemm_b128(A, B, D=wide[4:54, 8:80], config=cfg)
    ref = og.gemm(av[None], bv[None], d_fmt=formats.BF16)
    check(wide[4:54, 8:80].reshape(1, 50, 72), ref["D"], ref["bound"], formats.BF16)
    wide[4:54, 8:80] = 3.0
    assert (wide == 3.0).all()
    if tile_n == 64:
        return
    codes = torch.full((60, 128), 0x5A, dtype=torch.uint8, device=DEV)
    scales = torch.full((60, 3), 5.0, device=DEV)
    q = gge.B128Tensor(codes[4:54, 16:88].view(torch.float8_e4m3fn), scales[4:54, 1:2])
    gge.gge_gemm_b128(A, B, D=q, config=cfg)
    _check_q(q, ref["v"][0], 1e-5 * ref["bound"][0])
    codes[4:54, 16:88] = 0x5A
    scales[4:54, 1:2] = 5.0
    assert (codes == 0x5A).all() and (scales == 5.0).all()


# ------------------------------------------------------- backward activation epilogue

@pytest.mark.parametrize("act", ["relu", "gelu_tanh", "silu", "relu_sq"])
@pytest.mark.parametrize("tile_n", [0, 256, 128])
@pytest.mark.parametrize("pre", [torch.bfloat16, torch.float32, "e4m3", "e5m2"])
def test_dact(act, tile_n, pre):
    m, n, k = 140, 264, 300
    (A, av), (B, bv) = _held(_x(m, k, seed=1)), _held(_x(n, k, seed=2), 128)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(m, n, generator=g)
    if isinstance(pre, str):
        X, xv = _held(x, 1, pre)
    else:
        X = x.to(pre).to(DEV)
        xv = dec(X)
    ref = og.gemm_dact(av[None], bv[None], xv[None], act=act)
    want = activations.apply(act, xv)
    slack = np.abs(xv) * 2.0 ** -20
    for d, p in ((torch.bfloat16, torch.float32), ("e4m3", "e4m3"), (torch.float16, None)):
        D = _empty(m, n, 1, d) if isinstance(d, str) else torch.empty(m, n, dtype=d, device=DEV)
        P = None if p is None else _empty(m, n, 1, p) if isinstance(p, str) else torch.empty(m, n, dtype=p, device=DEV)
        gge.gge_gemm_b128_dact(A, B, X, D, act, PostAct=P, config=gge.make_config(tile_n=tile_n))
        assert _status() == "GGE_OK"
        if isinstance(d, str):
            _check_q(D, ref["v"][0], 1e-5 * ref["bound"][0])
        else:
            check(D[None], formats.round_to(ref["v"], FMT[d]), ref["bound"], FMT[d])
        if isinstance(p, str):
            _check_q(P, want, slack)
        elif P is not None:
            r = formats.round_to(want, FMT[p])
            assert (np.abs(dec(P) - r) <= slack + formats.quantum(r, FMT[p])).all()


# ---------------------------------------------------------------- grouped rows

def _groups(sizes):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("tile_n", [0, 256, 128, 64])
@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("sizes", [[5], [0, 130, 1, 0, 255, 257, 0], [1] * 40, [300, 0, 0, 77]])
def test_grouped_rows(tile_n, b_rows, sizes):
    n, k, groups, total = 136, 300, len(sizes), sum(sizes)
    A, av = _held(_x(total + 7, k, seed=total))                 # (seven rows of no group)
    B, bv = _held(torch.stack([_x(n, k, seed=50 + g) for g in range(groups)]), b_rows)
    cu = _groups(sizes)
    D = torch.full((total + 7, n), 9.0, dtype=torch.float32, device=DEV)
    cfg = gge.make_config(tile_n=tile_n)
    gge.gge_gemm_b128_varlen_m(A, B, cu, D=D, config=cfg)
    assert _status() == "GGE_OK"
    ref = og.gemm_varlen_m(av, bv, cu.cpu().numpy())
    got = dec(D)
    assert (got[total:] == 9.0).all()
    assert (np.abs(got - ref["v"])[:total] <= (1e-5 * ref["bound"] + formats.quantum(ref["v"], formats.F32))[:total]).all()
    if tile_n == 64:
        return
    # 8-bit outputs, the activation, and the backward from the checkpoint
    Z, Q = _empty(total + 7, n), _empty(total + 7, n)
    gge.gge_gemm_b128_varlen_m(A, B, cu, D=Z, PostAct=Q, act="silu", config=cfg)
    assert _status() == "GGE_OK"
    v = ref["v"][:total]
    bound = ref["bound"][:total]
    _check_q(gge.B128Tensor(Z.codes[:total], Z.scales[:total]), v, 1e-5 * bound)
    _check_q(gge.B128Tensor(Q.codes[:total], Q.scales[:total]), activations.apply("silu", v), _slack("silu", v, bound))
    assert (Z.codes[total:].contiguous().view(torch.uint8) == 0xA5).all() and torch.isnan(Z.scales[total:]).all()
    G = torch.full((total + 7, n), 9.0, dtype=torch.bfloat16, device=DEV)
    gge.gge_gemm_b128_dact(A, B, Z, G, "silu", cu_seqlens_m=cu, config=cfg)
    assert _status() == "GGE_OK"
    x = _numbers(gge.B128Tensor(Z.codes[:total], Z.scales[:total]))
    want = activations.DFN["silu"](x) * v
    tol = (np.abs(activations.DFN["silu"](x)) * 1e-5 + 1e-6) * bound + formats.quantum(want, formats.BF16)
    assert (np.abs(dec(G)[:total] - want) <= tol).all() and (dec(G)[total:] == 9.0).all()


@pytest.mark.parametrize("cu", [[0, 40, 30, 64], [0, 40, 200, 64], [-3, 20, 40, 64]])
def test_bad_offsets_are_reported(cu):
    A, B = _held(_x(64, 200))[0], _held(torch.stack([_x(72, 200, seed=g) for g in range(3)]), 128)[0]
    wide = torch.full((80, 72), 3.0, dtype=torch.bfloat16, device=DEV)
    gge.gge_gemm_b128_varlen_m(A, B, torch.tensor(cu, dtype=torch.int32, device=DEV), D=wide[8:72])
    assert _status() == "GGE_ERR_INDEX_RANGE"
    assert (wide[:8] == 3.0).all() and (wide[72:] == 3.0).all()


# ------------------------------------------------------------- streams, graphs, limits

@pytest.mark.parametrize("tile_n,splits", [(256, False), (128, False), (64, False), (64, True)])
def test_wait_timeout_reported_and_context_survives(tile_n, splits):
    A, B = gge.b128_empty(40, 4096, device=DEV), gge.b128_empty(256, 4096, 128, device=DEV)
    for q in (A, B):
        q.codes.view(torch.uint8).zero_()
        q.scales.zero_()
    D = torch.empty(40, 256, dtype=torch.bfloat16, device=DEV)
    cfg = gge.make_config(tile_n=tile_n, flags=2 | (0 if splits else 32), timeout_ns=20_000_000)
    gge.gge_gemm_b128(A, B, D=D, config=cfg)
    torch.cuda.synchronize()
    status, where, _ = gge.gge_read_device_status()
    # (a block's sum that is never handed on stops every role: whichever waits first says so --
    # loads 0, MMAs 1 and 2, sums 3, scales 10)
    assert status == "GGE_ERR_TIMEOUT" and where in (0, 1, 2, 3, 10)
    assert gge.gge_read_device_status()[0] == "GGE_OK"
    _product(40, 256, 4096, config=gge.make_config(tile_n=tile_n))


def test_streams_and_graphs():
    """Two streams at once with workspaces of their own; a captured chain replays with new data."""
    (A, av), (B, bv) = _held(_x(100, 1100, seed=11)), _held(_x(520, 1100, seed=12), 128)
    ref = og.gemm(av[None], bv[None], d_fmt=formats.BF16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = [gge.new_workspace(DEV) for _ in range(2)]
    D = [torch.empty(100, 520, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, w, d in zip(streams, work, D):
            with torch.cuda.stream(s):
                gge.gge_gemm_b128(A, B, D=d, workspace=w)
    torch.cuda.synchronize()
    for d in D:
        check(d[None], ref["D"], ref["bound"], formats.BF16)
    x = _x(100, 1100, seed=13, spread=0.5).to(DEV)
    q, z = _empty(100, 1100), _empty(100, 520)

    def chain(out):
        gge.gge_b128_quantize(x, q)
        gge.gge_gemm_b128(q, B, D=z)
        gge.gge_b128_dequantize(z, out)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(D[0])
    graph.replay()
    first = D[0].clone()
    x.mul_(0.5)
    graph.replay()
    chain(D[1])
    torch.cuda.synchronize()
    assert torch.equal(D[0], D[1]) and not torch.equal(first, D[1])


def test_arguments_refused():
    A, B = gge.b128_empty(40, 256, device=DEV), gge.b128_empty(64, 256, 128, device=DEV)
    D = torch.empty(40, 64, device=DEV)
    with pytest.raises(ValueError):
        gge.B128Tensor(A.codes, A.scales, 128)
    with pytest.raises(TypeError):
        gge.B128Tensor(A.codes.view(torch.uint8), A.scales)
    with pytest.raises(ValueError):
        gge.B128Tensor(A.codes.t(), A.scales.t())
    with pytest.raises(ValueError):
        gge.gge_gemm_b128_varlen_m(A, B, torch.zeros(2, dtype=torch.int64, device=DEV), D=D)
    with pytest.raises(gge.GgeError):
        gge.gge_gemm_b128(A, B)
    with pytest.raises(gge.GgeError):
        gge.gge_gemm_b128(A, B, D=gge.b128_empty(40, 64, 128, device=DEV))
    with pytest.raises(gge.GgeError):
        gge.gge_gemm_b128(A, B, D=gge.b128_empty(40, 64, device=DEV), config=gge.make_config(tile_n=64))
    with pytest.raises(TypeError):
        gge.gge_b128_quantize(D, D)
