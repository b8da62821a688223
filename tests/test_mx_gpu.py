"""Microscaled quantisation and the block-scaled product on the GPU against the
float64 oracle.

Quantisation is exact (codes and scales have to be equal); products are compared
within 1e-5 * sum |a b| + 1 ulp of the output, the bound of the other products
(the codes' products are exact, so only the fp32 sum differs).  gelu_tanh and silu add
2^-20 of the value they are taken of: their exponential and reciprocal are the SFU's
(2^-22 each), and with C that value may be large where sum |a b| is nothing."""

import numpy as np
import pytest
import torch

from grouped_gemm_epilogues_gb300 import binding as gge
from oracle import activations, formats, gemm as og, lowp

from helpers import FMT, check, dec

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
FORMATS = ("mxfp8", "mxfp4", "nvfp4")


def _x(rows, cols, dtype, seed=0, spread=3.0):
    """Values whose blocks differ in size, with zero, tiny and repeated ones."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(spread * torch.randn(rows, 1, generator=g).clamp(-2, 2))
    x[torch.rand(rows, cols, generator=g) < 0.05] = 0.0
    if rows > 2:
        x[1] = 0.0
    return x.to(dtype)


def _tscale(x):
    return (x.float().abs().max() / 2688.0).clamp_min(1e-20).reshape(1).to(DEV)


def _quantised(x, fmt, transposed=False, values=None):
    """Quantise a CPU matrix on the GPU: (MxTensor, values)."""
    t = _tscale(x) if fmt == "nvfp4" else None
    src = x.t().contiguous().to(DEV).t() if transposed else x.to(DEV)
    q = gge.mx_empty(*x.shape, fmt, device=DEV, tensor_scale=t)
    q.codes.fill_(0xA5)
    q.scales.fill_(0xA5)
    v = torch.full(x.shape, 7.0, dtype=values, device=DEV) if values else None
    gge.gge_mx_quantize(src, q, values=v)
    return q, v


def _check_codes(x, q, fmt):
    rows, cols = x.shape
    t = float(q.tensor_scale.cpu()) if q.tensor_scale is not None else 1.0
    ref, byte = lowp.quantise(dec(x), fmt, t)
    codes, flat = q.codes.cpu().numpy(), q.scales.cpu().numpy()
    got_byte, padding = lowp.scale_bytes(flat, rows, cols, fmt)
    assert np.array_equal(got_byte, byte)
    assert not padding.any(), "padding of the last scale word"
    got = lowp.decode(codes, flat, rows, cols, fmt, t)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[~np.isnan(ref)], ref[~np.isnan(ref)])
    # the codes past the last column are zero
    per = 8 if fmt == "mxfp8" else 4
    tail = np.unpackbits(codes, axis=1, bitorder="little")[:, cols * per:]
    assert not tail.any()
    return ref


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 31), (7, 33), (130, 64), (64, 257), (65, 129),
                                       (5, 1000), (129, 2049)])
def test_quantise_is_exact(fmt, transposed, rows, cols):
    dtype = (torch.bfloat16, torch.float16, torch.float32)[(rows + cols) % 3]
    x = _x(rows, cols, dtype, seed=rows)
    q, v = _quantised(x, fmt, transposed, torch.float32)
    ref = _check_codes(x, q, fmt)
    assert np.array_equal(dec(v), formats.round_to(ref, formats.F32))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("values", [torch.bfloat16, torch.float16, torch.float32])
def test_quantise_values_types_and_round_trip(fmt, transposed, values):
    x = _x(70, 301, torch.bfloat16, seed=4, spread=0.5)
    q, v = _quantised(x, fmt, transposed, values)
    ref = _check_codes(x, q, fmt)
    # nvfp4's third factor rounds the fp32 value before the 16-bit one
    want = formats.round_to(formats.round_to(ref, formats.F32), FMT[values])
    assert np.array_equal(dec(v), want)
    y = torch.empty(70, 301, dtype=values, device=DEV)
    gge.gge_mx_dequantize(q, y)
    assert np.array_equal(dec(y), want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("transposed", [False, True])
def test_quantise_extremes_and_not_finite(fmt, transposed):
    x = torch.zeros(140, 96)
    x[0, :32] = 3.0e38
    x[1, :32] = 2.0 ** -140
    x[2, 0], x[2, 40], x[3, 95] = float("inf"), float("-inf"), float("nan")
    x[4] = torch.linspace(-1, 1, 96)
    x[139] = 448.0
    t = torch.ones(1, device=DEV) if fmt == "nvfp4" else None
    src = x.t().contiguous().to(DEV).t() if transposed else x.to(DEV)
    q = gge.mx_empty(140, 96, fmt, device=DEV, tensor_scale=t)
    gge.gge_mx_quantize(src, q)
    _check_codes(x, q, fmt)


def test_quantise_strided_rows_batches_and_guards():
    """Rows that start on odd elements and are longer than the matrix, batches, and the bytes
    beside every output row."""
    g = torch.Generator().manual_seed(2)
    big = torch.randn(3, 40, 211, generator=g).bfloat16().to(DEV)
    x = big[:, 1:38, 3:202]                                   # 37 rows of 199, misaligned
    rows, cols, fmt = 37, 199, "mxfp4"
    row = gge._mx_row_bytes(1, cols)
    wide = torch.full((3, rows, row + 48), 0x5A, dtype=torch.uint8, device=DEV)
    scales = torch.empty(3 * gge._mx_scale_bytes(1, rows, cols), dtype=torch.uint8, device=DEV)
    q = gge.MxTensor(wide[:, :, :row], scales, fmt, rows, cols)
    vals = torch.full((3, rows, cols + 9), 5.0, dtype=torch.float16, device=DEV)
    gge.gge_mx_quantize(x, q, values=vals[:, :, 5:5 + cols])
    assert (wide[:, :, row:] == 0x5A).all()
    assert (vals[:, :, :5] == 5.0).all() and (vals[:, :, 5 + cols:] == 5.0).all()
    per = scales.numel() // 3
    for b in range(3):
        one = gge.MxTensor(wide[b, :, :row], scales[b * per:(b + 1) * per], fmt, rows, cols)
        ref = _check_codes(x[b].cpu(), one, fmt)
        assert np.array_equal(dec(vals[b, :, 5:5 + cols]), formats.round_to(ref, formats.F16))


def test_quantise_past_32_bits_of_elements():
    """The last rows of a matrix of more than 2^31 elements."""
    rows, cols = 70_000, 32_768
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    tail = _x(5, cols, torch.bfloat16, seed=9).to(DEV)
    x[-5:] = tail
    q = gge.mx_empty(rows, cols, "mxfp8", device=DEV)
    gge.gge_mx_quantize(x, q)
    y = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    gge.gge_mx_dequantize(q, y)
    assert np.array_equal(dec(y[-5:]), lowp.quantise(dec(tail), "mxfp8")[0])
    assert not y[:-5].any()


# ---------------------------------------------------------------- products

def _operands(m, n, k, fmt, seed, batch=None):
    out = []
    for rows, s in ((m, seed), (n, seed + 1)):
        xs = [_x(rows, k, torch.bfloat16, s + 10 * b, spread=0.7) for b in range(batch or 1)]
        t = max(float(_tscale(x).cpu()) for x in xs)
        t = torch.tensor([t], device=DEV) if fmt == "nvfp4" else None
        q = gge.mx_empty(rows, k, fmt, device=DEV, batch=batch, tensor_scale=t)
        # (what no call may read: the scales of rows past the last one)
        q.scales.fill_(0xFF)
        gge.gge_mx_quantize(torch.stack(xs).to(DEV) if batch else xs[0].to(DEV), q)
        tv = float(t.cpu()) if t is not None else 1.0
        codes, flat = q.codes.cpu().numpy(), q.scales.cpu().numpy()
        if batch:
            per = flat.size // batch
            vals = np.stack([lowp.decode(codes[b], flat[b * per:(b + 1) * per], rows, k, fmt, tv)
                             for b in range(batch)])
        else:
            vals = lowp.decode(codes, flat, rows, k, fmt, tv)[None]
        out.append((q, vals))
    return out


def _check_product(m, n, k, fmt, act="none", with_c=False, d=torch.bfloat16, p=torch.bfloat16, alpha=1.0,
                   beta=0.0, batch=None, config=None, dev_scalars=False, seed=0, both=True):
    (A, av), (B, bv) = _operands(m, n, k, fmt, seed, batch)
    shape = (batch, m, n) if batch else (m, n)
    g = torch.Generator().manual_seed(seed + 99)
    C = torch.randn(shape, generator=g).to(d) if with_c else None
    D = torch.full(shape, float("nan"), dtype=d, device=DEV) if both or act == "none" else None
    P = torch.full(shape, float("nan"), dtype=p, device=DEV) if act != "none" else None
    kw = dict(alpha=alpha, beta=beta)
    if dev_scalars:
        kw = dict(alpha=99.0, beta=99.0, alpha_dev=torch.tensor([alpha], device=DEV),
                  beta_dev=torch.tensor([beta], device=DEV))
    gge.gge_gemm_mx(A, B, D=D, C=C.to(DEV) if with_c else None, PostAct=P, act=act, config=config, **kw)
    torch.cuda.synchronize()
    assert gge.gge_read_device_status()[0] == "GGE_OK"
    # (a sum over no K is an empty product)
    ref = og.gemm(av, bv, dec(C).reshape(batch or 1, m, n) if with_c else None, alpha=alpha, beta=beta,
                  act=act, d_fmt=FMT[d], p_fmt=FMT[p])
    if D is not None:
        check(D.reshape(ref["D"].shape), ref["D"], ref["bound"], FMT[d], "none", "D")
    if P is not None:
        bound = ref["bound"] + (np.abs(ref["v"]) * 2.0 ** -20 / 1e-5 if act in ("gelu_tanh", "silu") else 0.0)
        check(P.reshape(ref["P"].shape), ref["P"], bound, FMT[p], act, "PostAct", x=ref["v"])
    return D, P


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m,n,k", [(1, 8, 1), (1, 264, 200), (2, 72, 31), (16, 512, 1024), (63, 136, 96),
                                   (64, 128, 33), (65, 128, 640), (127, 200, 257), (129, 264, 512),
                                   (300, 520, 1100), (257, 8, 2080)])
def test_product_shapes(fmt, m, n, k):
    _check_product(m, n, k, fmt, seed=m)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tile_n", [256, 128, 64])
@pytest.mark.parametrize("m,n,k", [(300, 520, 1100), (70, 264, 4000), (600, 1032, 300)])
def test_every_tile_shape(fmt, tile_n, m, n, k):
    """Each tile shape on the same problems, whole (one or several tiles a CTA) and, where
    the shape allows it, split along K over a cluster."""
    for kw in (dict(), dict(flags=32), dict(num_ctas=4), dict(flags=32 | 8), dict(flags=128, raster_band=2),
               dict(stages=2)):
        _check_product(m, n, k, fmt, "silu", config=gge.make_config(tile_n=tile_n, **kw), seed=tile_n)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m,n,k", [(16, 128, 8192), (16, 1024, 8192), (40, 4096, 4096), (100, 256, 8192),
                                   (128, 2048, 2048)])
def test_split_k_clusters(fmt, m, n, k):
    """Few tiles and a long K: the tile's sum comes from several CTAs.  Calls repeat bit for bit."""
    first = _check_product(m, n, k, fmt, "gelu_tanh", True, beta=0.5, seed=3)
    again = _check_product(m, n, k, fmt, "gelu_tanh", True, beta=0.5, seed=3)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("act", ["relu", "gelu_tanh", "silu", "relu_sq"])
@pytest.mark.parametrize("tile_n", [256, 128, 64])
def test_epilogues(act, tile_n):
    cfg = gge.make_config(tile_n=tile_n)
    _check_product(130, 264, 520, "mxfp8", act, True, torch.float32, torch.float16, 0.75, -0.5, config=cfg)
    _check_product(130, 264, 520, "nvfp4", act, True, torch.float16, torch.float32, 0.75, 0.5, config=cfg,
                   dev_scalars=True)
    _check_product(130, 264, 520, "mxfp4", act, False, both=False, config=cfg)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tile_n", [0, 256, 128, 64])
def test_batches(fmt, tile_n):
    _check_product(70, 136, 300, fmt, with_c=True, beta=1.0, batch=3, config=gge.make_config(tile_n=tile_n))


def test_no_k_and_empty_sides():
    for fmt in FORMATS:
        A, B = gge.mx_empty(40, 0, fmt, device=DEV), gge.mx_empty(64, 0, fmt, device=DEV)
        C = torch.randn(40, 64, device=DEV).bfloat16()
        D = torch.full_like(C, float("nan"))
        gge.gge_gemm_mx(A, B, D=D, C=C, beta=0.5)
        assert torch.equal(D, (C.float() * 0.5).bfloat16())
        A = gge.mx_empty(0, 96, fmt, device=DEV)
        gge.gge_gemm_mx(A, gge.mx_empty(64, 96, fmt, device=DEV), D=torch.empty(0, 64, device=DEV))
        gge.gge_mx_quantize(torch.empty(0, 96, device=DEV), A)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tile_n", [256, 128, 64])
def test_not_finite_rows_stay_in_their_rows(fmt, tile_n):
    """A NaN block of A makes its row of D NaN and no other; rows past the last one and the
    columns past the last one never reach an output."""
    x = _x(70, 200, torch.bfloat16, 5, spread=0.5)
    x[33, 100] = float("nan")
    y = _x(72, 200, torch.bfloat16, 6, spread=0.5)
    qs = []
    for t in (x, y):
        q = gge.mx_empty(*t.shape, fmt, device=DEV,
                         tensor_scale=torch.ones(1, device=DEV) if fmt == "nvfp4" else None)
        q.scales.fill_(0xFF)
        gge.gge_mx_quantize(t.to(DEV), q)
        qs.append(q)
    D = torch.empty(70, 72, dtype=torch.float32, device=DEV)
    gge.gge_gemm_mx(*qs, D=D, config=gge.make_config(tile_n=tile_n))
    bad = torch.isnan(D).cpu()
    assert bad[33].all() and not bad[torch.arange(70) != 33].any()


def test_output_guards_and_strides():
    for tile_n in (256, 128, 64):
        (A, av), (B, bv) = _operands(50, 72, 160, "mxfp8", 7)
        wide = torch.full((60, 96), 3.0, dtype=torch.bfloat16, device=DEV)
        gge.gge_gemm_mx(A, B, D=wide[4:54, 8:80], config=gge.make_config(tile_n=tile_n))
        ref = og.gemm(av, bv, d_fmt=formats.BF16)
        check(wide[4:54, 8:80].reshape(1, 50, 72), ref["D"], ref["bound"], formats.BF16)
        wide[4:54, 8:80] = 3.0
        assert (wide == 3.0).all()


@pytest.mark.parametrize("tile_n,splits", [(256, False), (128, False), (64, False), (64, True)])
def test_wait_timeout_reported_and_context_survives(tile_n, splits):
    A, B = (gge.mx_empty(r, 4096, "mxfp8", device=DEV) for r in (40, 256))
    for q in (A, B):
        q.codes.zero_()
        q.scales.zero_()
    D = torch.empty(40, 256, dtype=torch.bfloat16, device=DEV)
    cfg = gge.make_config(tile_n=tile_n, flags=2 | (0 if splits else 32), timeout_ns=20_000_000)
    gge.gge_gemm_mx(A, B, D=D, config=cfg)
    torch.cuda.synchronize()
    status, where, _ = gge.gge_read_device_status()
    assert status == "GGE_ERR_TIMEOUT" and where == 3
    assert gge.gge_read_device_status()[0] == "GGE_OK"
    _check_product(40, 256, 4096, "mxfp8", config=gge.make_config(tile_n=tile_n))


def test_streams_and_graphs():
    """Two streams at once with workspaces of their own; a captured call replays with new data."""
    (A, av), (B, bv) = _operands(100, 520, 1100, "nvfp4", 11)
    ref = og.gemm(av, bv, d_fmt=formats.BF16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = [gge.new_workspace(DEV) for _ in range(2)]
    D = [torch.empty(100, 520, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, w, d in zip(streams, work, D):
            with torch.cuda.stream(s):
                gge.gge_gemm_mx(A, B, D=d, workspace=w)
    torch.cuda.synchronize()
    for d in D:
        check(d[None], ref["D"], ref["bound"], formats.BF16)
    x = _x(100, 1100, torch.bfloat16, 12, spread=0.5).to(DEV)
    q = gge.mx_empty(100, 1100, "nvfp4", device=DEV, tensor_scale=_tscale(x))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gge.gge_mx_quantize(x, q)
        gge.gge_gemm_mx(q, B, D=D[0])
    graph.replay()
    first = D[0].clone()
    x.mul_(0.5)
    graph.replay()
    gge.gge_mx_quantize(x, q)
    gge.gge_gemm_mx(q, B, D=D[1])
    torch.cuda.synchronize()
    assert torch.equal(D[0], D[1]) and not torch.equal(first, D[1])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("act", ["relu", "gelu_tanh", "silu", "relu_sq"])
@pytest.mark.parametrize("m,n,k,tile_n", [(130, 264, 520, 256), (130, 264, 520, 128), (16, 136, 4096, 64),
                                          (100, 136, 4096, 0)])
def test_backward_activation_epilogue(fmt, act, m, n, k, tile_n):
    (A, av), (B, bv) = _operands(m, n, k, fmt, 21)
    g = torch.Generator().manual_seed(5)
    X = torch.randn(m, n, generator=g).bfloat16()
    D = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    P = torch.empty_like(D)
    gge.gge_gemm_mx_dact(A, B, X.to(DEV), D, act, PostAct=P, config=gge.make_config(tile_n=tile_n))
    ref = og.gemm_dact(av, bv, dec(X)[None], act=act, d_fmt=formats.BF16, p_fmt=formats.BF16)
    # act'(x) is evaluated in fp32 from the SFU's functions: 1e-6 of sum |a b| on top
    bound = ref["bound"] * (1.1 if act in ("gelu_tanh", "silu") else 1.0)
    check(D[None], ref["D"], bound, formats.BF16, what="D")
    pb = np.abs(dec(X)[None]) * 2.0 ** -20 / 1e-5
    check(P[None], ref["P"], pb, formats.BF16, what="PostAct")


def test_python_refusals():
    x = torch.randn(64, 128, device=DEV).bfloat16()
    q, q8 = gge.mx_empty(64, 128, "mxfp4", device=DEV), gge.mx_empty(64, 128, "mxfp8", device=DEV)
    with pytest.raises(gge.GgeError, match="GGE_ERR_INVALID_ARG"):
        gge.gge_mx_quantize(x[:63], q)
    with pytest.raises(gge.GgeError, match="GGE_ERR_UNSUPPORTED"):
        gge.gge_gemm_mx(q, q8, D=torch.empty(64, 64, device=DEV))
    with pytest.raises(ValueError, match="CUDA"):
        gge.gge_mx_quantize(x, q, values=x.cpu())
    with pytest.raises(ValueError, match="different devices"):
        gge.gge_mx_quantize(x.cpu(), q)
    with pytest.raises(TypeError, match="unsupported dtype"):
        gge.gge_mx_quantize(x.double(), q)
    with pytest.raises(TypeError, match="expected a tensor"):
        gge.gge_gemm_mx(q, q, D=3.0)
    with pytest.raises(ValueError, match="2-D"):
        gge.gge_mx_quantize(x[0], q)
    with pytest.raises(ValueError, match="contiguous"):
        gge.gge_rmsnorm(x, torch.ones(256, device=DEV)[::2].bfloat16()[:100], Y=torch.empty_like(x))
    with pytest.raises(ValueError, match="do not match"):
        gge.MxTensor(q.codes[:, :32], q.scales, "mxfp4", 64, 128)
    with pytest.raises(ValueError, match="do not match"):
        gge.MxTensor(q.codes, q.scales[:100], "mxfp4", 64, 128)
    with pytest.raises(TypeError):
        gge.MxTensor(q.codes.float(), q.scales, "mxfp4", 64, 128)
    with pytest.raises(KeyError):
        gge.mx_empty(4, 4, "fp6", device=DEV)
    with pytest.raises(ValueError, match="1 contiguous values"):
        gge.MxTensor(q.codes, q.scales, "mxfp4", 64, 128, tensor_scale=torch.ones(2, device=DEV))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tile_n", [256, 128, 64])
@pytest.mark.parametrize("k", [64, 500, 1300])
def test_many_short_tiles_a_cta(fmt, tile_n, k):
    """Many tiles of a short K on few CTAs, so that every wait between the accumulators is
    the one that decides: the outputs equal those of one tile a CTA bit for bit."""
    (A, _), (B, _) = _operands(500, 1496, k, fmt, 31)
    one = torch.empty(500, 1496, dtype=torch.bfloat16, device=DEV)
    gge.gge_gemm_mx(A, B, D=one, config=gge.make_config(tile_n=tile_n, flags=32))
    for ctas in (2, 4, 10):
        for _ in range(4):
            D = torch.full_like(one, float("nan"))
            gge.gge_gemm_mx(A, B, D=D, config=gge.make_config(tile_n=tile_n, num_ctas=ctas))
            assert torch.equal(D, one)
