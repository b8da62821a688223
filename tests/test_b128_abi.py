"""Refusals of the entry points on 8 bits with a scale for each block of 128, through the C ABI
(no GPU: a rejected call launches nothing), and the layout of the matrices that the binding makes."""

import ctypes

import pytest
import torch

from grouped_gemm_epilogues_gb300 import binding as b

INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4
P = 1 << 20          # an aligned address that is never dereferenced
BF16, F16, E4M3, F32, E5M2 = 0, 1, 2, 4, 3


@pytest.fixture(scope="module")
def lib():
    return b.load()


def tensor(rows=64, cols=128, dtype=BF16, ptr=P, batch=1, sr=None, sc=1, sb=None, reserved=0):
    return b.GgeTensor(ptr, dtype, reserved, rows, cols, batch, cols if sr is None else sr, sc,
                       rows * cols if sb is None else sb)


def b128(rows=64, cols=128, block=1, dtype=E4M3, codes=P, scales=P, batch=1, sr=None, sb=None, s_row=1, s_col=None,
         s_batch=None):
    row = (cols + 15) // 16 * 16
    blocks = (rows + max(block, 1) - 1) // max(block, 1)
    return b.GgeB128Tensor(codes, scales, dtype, block, rows, cols, batch, row if sr is None else sr,
                           rows * row if sb is None else sb, s_row, blocks if s_col is None else s_col,
                           blocks * ((cols + 127) // 128) if s_batch is None else s_batch)


def ref(s):
    return ctypes.addressof(s) if s is not None else None


def test_struct_layouts():
    """The sizes that a C compiler gives the header's structs on both 64-bit machines."""
    assert ctypes.sizeof(b.GgeB128Tensor) == 2 * 8 + 2 * 4 + 8 * 8
    assert ctypes.sizeof(b.GgeGemmB128Args) == 2 * 88 + 7 * 8 + 4 * 4 + 3 * 8
    assert ctypes.sizeof(b.GgeLayernormArgs) == 64 + 8 * 8 + 2 * 4 + 2 * 8
    assert ctypes.sizeof(b.GgeLayernormBwdArgs) == 2 * 64 + 4 * 8 + 2 * 4 + 4 * 8


BAD_MATRICES = [
    (dict(dtype=BF16), UNSUPPORTED), (dict(block=64), UNSUPPORTED), (dict(block=0), UNSUPPORTED),
    (dict(batch=0), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(codes=P + 8), ALIGNMENT), (dict(scales=P + 2), ALIGNMENT), (dict(sr=112), INVALID),
    (dict(sr=136), ALIGNMENT), (dict(s_row=-1), INVALID), (dict(s_col=-1), INVALID),
]


@pytest.mark.parametrize("kw,code", BAD_MATRICES + [
    (dict(s_row=0), INVALID), (dict(cols=256, s_col=0), INVALID), (dict(cols=256, s_col=63), INVALID),
    (dict(rows=63), INVALID), (dict(cols=120), INVALID)])
def test_quantize_refuses_the_output(lib, kw, code):
    cols = kw.get("cols", 128)
    x = tensor(64, cols if cols != 120 else 128)
    assert lib.gge_b128_quantize(ref(x), ref(b128(**kw)), None, None) == code


@pytest.mark.parametrize("x,v,code", [
    (None, None, INVALID), (tensor(dtype=E4M3), None, UNSUPPORTED), (tensor(reserved=1), None, INVALID),
    (tensor(ptr=None), None, INVALID), (tensor(ptr=P + 1), None, ALIGNMENT), (tensor(sr=300, sc=2), None, UNSUPPORTED),
    (tensor(sr=-5), None, INVALID), (tensor(), tensor(cols=120), INVALID), (tensor(), tensor(sr=100), INVALID),
    (tensor(), tensor(dtype=E4M3), UNSUPPORTED), (tensor(), tensor(sr=1, sc=64), UNSUPPORTED),
])
def test_quantize_refuses_the_input(lib, x, v, code):
    assert lib.gge_b128_quantize(ref(x), ref(b128()), ref(v), None) == code


@pytest.mark.parametrize("kw,code", BAD_MATRICES)
def test_inputs_in_8_bits(lib, kw, code):
    x = b128(**kw)
    assert lib.gge_b128_transpose(ref(x), ref(b128(128, 64)), None, None) == code
    assert lib.gge_b128_dequantize(ref(x), ref(tensor()), None) == code
    assert product(lib, A=x) == code
    assert product(lib, B=x, D=tensor(64, 64)) == code
    assert norm_bwd(lib, h=None, h8=x) == code


def test_inputs_may_share_scales(lib):
    """One scale for all rows is a stride of zero: fine to read, not to write."""
    shared = b128(0, 128, s_row=0)
    assert lib.gge_b128_dequantize(ref(shared), ref(tensor(0, 128)), None) == 0
    assert lib.gge_b128_quantize(ref(tensor()), ref(b128(s_row=0)), None, None) == INVALID


@pytest.mark.parametrize("q,code", [(b128(64, 128), INVALID), (b128(128, 63), INVALID), (None, INVALID)])
def test_transpose_refusals(lib, q, code):
    assert lib.gge_b128_transpose(ref(b128()), ref(q), None, None) == code
    assert lib.gge_b128_transpose(None, ref(b128()), None, None) == INVALID


@pytest.mark.parametrize("y,code", [(None, INVALID), (tensor(rows=65), INVALID), (tensor(sr=64), INVALID),
                                    (tensor(sr=1, sc=64), UNSUPPORTED), (tensor(dtype=E4M3), UNSUPPORTED)])
def test_dequantize_refusals(lib, y, code):
    assert lib.gge_b128_dequantize(ref(b128()), ref(y), None) == code


def product(lib, A=None, B=None, C=None, D=tensor(64, 72), P_=None, C8=None, D8=None, P8=None, cu=None, groups=0, act=0,
            config=None, ws=P, n=256, dact=False):
    A = A if A is not None else b128(64, 128)
    B = B if B is not None else b128(72, 128, 128)
    args = b.GgeGemmB128Args(A, B, ref(C), ref(D), ref(P_), ref(C8), ref(D8), ref(P8), cu, groups, act, 1.0, 0.0, None,
                             None, ref(config))
    fn = lib.gge_gemm_b128_dact if dact else lib.gge_gemm_b128
    return fn(ref(args), ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=None), INVALID), (dict(act=9), INVALID), (dict(act=1), INVALID),
    (dict(B=b128(72, 96, 128)), INVALID), (dict(A=b128(64, 128, batch=2)), INVALID), (dict(A=b128(63, 128)), INVALID),
    (dict(B=b128(68, 128, 128), D=tensor(64, 68, sr=72)), UNSUPPORTED),
    (dict(D=tensor(64, 72, sr=73)), ALIGNMENT), (dict(D=tensor(64, 72, ptr=P + 8)), ALIGNMENT),
    (dict(D=tensor(64, 72, sr=64)), INVALID), (dict(D=tensor(64, 72, dtype=E4M3)), UNSUPPORTED),
    (dict(C=tensor(64, 80)), INVALID), (dict(n=128), WORKSPACE), (dict(ws=P + 4), ALIGNMENT),
    # both forms of one matrix, 8-bit forms of the wrong shape or blocks
    (dict(D8=b128(64, 72)), INVALID), (dict(D=None, D8=b128(64, 80)), INVALID),
    (dict(D=None, D8=b128(64, 72, 128)), UNSUPPORTED), (dict(C8=b128(64, 72, 128)), UNSUPPORTED),
    (dict(C=tensor(64, 72), C8=b128(64, 72)), INVALID), (dict(P_=tensor(64, 72), P8=b128(64, 72)), INVALID),
    (dict(D=None, D8=b128(64, 72, s_row=0)), INVALID),
    # groups
    (dict(groups=-1), INVALID), (dict(groups=2), INVALID), (dict(cu=P), INVALID), (dict(cu=P, groups=1025), UNSUPPORTED),
    (dict(cu=P + 2, groups=2), ALIGNMENT), (dict(cu=P, groups=2), INVALID),
    (dict(cu=P, groups=2, A=b128(64, 128, batch=2), B=b128(72, 128, 128, batch=2)), INVALID),
    # shapes that there are not
    (dict(config=b.make_config(tile_n=192)), UNSUPPORTED), (dict(config=b.make_config(stages=1)), UNSUPPORTED),
    (dict(config=b.make_config(flags=4)), UNSUPPORTED), (dict(config=b.make_config(cta_group=2)), UNSUPPORTED),
    (dict(config=b.make_config(tile_n=64), D=None, D8=b128(64, 72)), UNSUPPORTED),
    # the backward: C, D and an activation; C is read again after D is written
    (dict(dact=True, act=3), INVALID), (dict(dact=True, C=tensor(64, 72, ptr=2 * P)), INVALID),
    (dict(dact=True, C=tensor(64, 72, ptr=2 * P), act=3, D=None, P_=tensor(64, 72)), INVALID),
    (dict(dact=True, C=tensor(64, 72), act=3), INVALID),
    (dict(dact=True, C=tensor(64, 72, ptr=2 * P), act=3, P_=tensor(64, 72, ptr=2 * P)), INVALID),
    (dict(dact=True, C8=b128(64, 72), act=3, D=None, D8=b128(64, 72)), INVALID),
])
def test_product_refusals(lib, kw, code):
    assert product(lib, **kw) == code


def norm(lib, x=tensor(), residual=None, out=None, y=tensor(), q=None, values=None, h8=None, weight=P, bias=P, pt=BF16,
         mean=P, rstd=P):
    args = b.GgeLayernormArgs(x, ref(residual), ref(out), ref(y), ref(q), ref(values), ref(h8), weight, bias, pt, 1e-5,
                              mean, rstd)
    return lib.gge_layernorm(ref(args), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=tensor(batch=2)), UNSUPPORTED), (dict(x=tensor(dtype=E4M3)), UNSUPPORTED),
    (dict(x=tensor(sr=1, sc=64)), UNSUPPORTED), (dict(pt=E4M3), UNSUPPORTED), (dict(weight=P + 1), ALIGNMENT),
    (dict(bias=P + 1), ALIGNMENT), (dict(mean=P + 2), ALIGNMENT), (dict(rstd=P + 2), ALIGNMENT),
    (dict(y=tensor(dtype=F16)), UNSUPPORTED), (dict(y=tensor(rows=60)), INVALID), (dict(y=tensor(sr=100)), INVALID),
    (dict(residual=tensor(dtype=F32)), UNSUPPORTED), (dict(out=tensor()), INVALID),
    (dict(residual=tensor(), out=tensor(sr=100)), INVALID), (dict(values=tensor()), INVALID),
    (dict(q=b128(64, 96)), INVALID), (dict(q=b128(block=128)), UNSUPPORTED), (dict(h8=b128(block=128)), UNSUPPORTED),
    (dict(q=b128(), values=tensor(cols=96)), INVALID), (dict(q=b128(s_row=0)), INVALID),
    (dict(h8=b128(codes=P + 4)), ALIGNMENT), (dict(q=b128(batch=2)), INVALID),
])
def test_norm_refusals(lib, kw, code):
    assert norm(lib, **kw) == code


def norm_bwd(lib, dy=tensor(), h=tensor(), h8=None, dh=None, dx=tensor(), weight=P, wt=BF16, reserved=0, mean=P, rstd=P,
             dw=None, db=None, ws=None, n=0):
    args = b.GgeLayernormBwdArgs(dy, ref(h), ref(h8), ref(dh), dx, weight, wt, reserved, mean, rstd, dw, db)
    return lib.gge_layernorm_bwd(ref(args), ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(reserved=1), INVALID), (dict(h=None), INVALID), (dict(h8=b128()), INVALID), (dict(mean=None), INVALID),
    (dict(rstd=None), INVALID), (dict(dy=tensor(batch=2)), UNSUPPORTED), (dict(h=tensor(dtype=F16)), UNSUPPORTED),
    (dict(h=tensor(rows=63)), INVALID), (dict(dh=tensor(cols=120)), INVALID), (dict(dx=tensor(sr=100)), INVALID),
    (dict(dx=tensor(dtype=F32)), UNSUPPORTED), (dict(wt=E4M3), UNSUPPORTED), (dict(weight=P + 1), ALIGNMENT),
    (dict(rstd=P + 2), ALIGNMENT), (dict(h=None, h8=b128(63, 128)), INVALID),
])
def test_norm_backward_refusals(lib, kw, code):
    assert norm_bwd(lib, **kw) == code


def test_null_arguments(lib):
    assert lib.gge_b128_quantize(None, None, None, None) == INVALID
    assert lib.gge_gemm_b128(None, P, 256, None) == INVALID
    assert lib.gge_gemm_b128_dact(None, P, 256, None) == INVALID
    assert lib.gge_layernorm(None, None) == INVALID
    assert lib.gge_layernorm_bwd(None, None, 0, None) == INVALID


def test_empty_calls_do_nothing(lib):
    x, q = tensor(0, 128, ptr=None), b128(0, 128, codes=None, scales=None)
    assert lib.gge_b128_quantize(ref(x), ref(q), None, None) == 0
    assert lib.gge_b128_dequantize(ref(q), ref(x), None) == 0
    assert lib.gge_b128_transpose(ref(q), ref(b128(128, 0, codes=None, scales=None)), None, None) == 0
    assert norm(lib, x=x, y=x) == 0
    assert norm_bwd(lib, dy=x, h=x, dx=x, mean=None, rstd=None) == 0
    assert product(lib, A=q, D=tensor(0, 72, ptr=None)) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,block,batch", [(1, 1, 1, None), (129, 257, 128, None), (7, 100, 1, 3), (0, 64, 1, None),
                                                   (300, 128, 128, 2)])
def test_empty_matrix_has_its_layout(rows, cols, block, batch):
    q = b.b128_empty(rows, cols, block, device="cuda", batch=batch)
    lead = (batch,) if batch else ()
    assert tuple(q.codes.shape) == lead + (rows, cols) and q.codes.dtype == torch.float8_e4m3fn
    assert q.codes.stride(-1) == 1 and (rows < 2 or q.codes.stride(-2) % 16 == 0)
    assert tuple(q.scales.shape) == lead + (-(-rows // block), -(-cols // 128)) and q.scales.dtype == torch.float32
    if q.scales.shape[-2] > 1:      # a column block's scales lie together
        assert q.scales.stride(-2) == 1
    assert b.b128_empty(4, 64, dtype=torch.float8_e5m2, device="cuda").codes.dtype == torch.float8_e5m2
