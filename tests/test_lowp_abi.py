"""Refusals and host-side helpers of the low-precision entry points, through the C ABI
(no GPU: a rejected call launches nothing)."""

import ctypes

import pytest

from grouped_gemm_epilogues_gb300 import binding as b

INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4
P = 1 << 20          # an aligned address that is never dereferenced
BF16, F16, E4M3, F32 = 0, 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    return b.load()


def tensor(rows=64, cols=128, dtype=BF16, ptr=P, batch=1, sr=None, sc=1, sb=None, reserved=0):
    return b.GgeTensor(ptr, dtype, reserved, rows, cols, batch, cols if sr is None else sr, sc,
                       rows * cols if sb is None else sb)


def mx(rows=64, cols=128, fmt=0, codes=P, scales=P, t=None, batch=1, sr=None, reserved=0, sb=None, ss=None):
    row = b._mx_row_bytes(fmt, cols) if 0 <= fmt <= 2 else 128
    per = b._mx_scale_bytes(fmt, rows, cols) if 0 <= fmt <= 2 else 512
    return b.GgeMxTensor(codes, scales, t, fmt, reserved, rows, cols, batch, row if sr is None else sr,
                         rows * row if sb is None else sb, per if ss is None else ss)


def ref(s):
    return ctypes.addressof(s) if s is not None else None


def test_sizes(lib):
    for i, name in enumerate(("mxfp8", "mxfp4", "nvfp4")):
        assert b.MX_FORMAT[name] == i
        for rows, cols in ((1, 1), (128, 32), (129, 33), (7, 4096), (0, 5), (300, 0)):
            assert lib.gge_mx_row_bytes(i, cols) == b._mx_row_bytes(i, cols)
            assert lib.gge_mx_scale_bytes(i, rows, cols) == b._mx_scale_bytes(i, rows, cols)
    assert lib.gge_mx_row_bytes(0, 33) == 64 and lib.gge_mx_row_bytes(2, 33) == 32
    assert lib.gge_mx_scale_bytes(2, 129, 65) == 2 * 2 * 512
    assert lib.gge_mx_row_bytes(3, 64) == 0 and lib.gge_mx_scale_bytes(-1, 64, 64) == 0


def test_struct_layouts():
    """The sizes that a C compiler gives the header's structs on both 64-bit machines."""
    assert ctypes.sizeof(b.GgeTensor) == 64 and ctypes.sizeof(b.GgeMxTensor) == 80
    assert ctypes.sizeof(b.GgeGemmMxArgs) == 2 * 80 + 3 * 8 + 8 + 2 * 8 + 8 + 8
    assert ctypes.sizeof(b.GgeRmsnormArgs) == 64 + 6 * 8 + 8 + 8
    assert ctypes.sizeof(b.GgeRmsnormBwdArgs) == 3 * 64 + 8 + 8 + 8 + 2 * 8


@pytest.mark.parametrize("x,q,v,code", [
    (None, mx(), None, INVALID), (tensor(), None, None, INVALID),
    (tensor(dtype=E4M3), mx(), None, UNSUPPORTED), (tensor(reserved=1), mx(), None, INVALID),
    (tensor(ptr=None), mx(), None, INVALID), (tensor(ptr=P + 1), mx(), None, ALIGNMENT),
    (tensor(sr=300, sc=2), mx(), None, UNSUPPORTED), (tensor(rows=63), mx(), None, INVALID),
    (tensor(sr=-5), mx(), None, INVALID), (tensor(), mx(fmt=3), None, INVALID),
    (tensor(), mx(fmt=0, t=P), None, INVALID), (tensor(), mx(fmt=2, t=P + 2), None, ALIGNMENT),
    (tensor(), mx(codes=None), None, INVALID), (tensor(), mx(scales=None), None, INVALID),
    (tensor(), mx(codes=P + 8), None, ALIGNMENT), (tensor(), mx(scales=P + 64), None, ALIGNMENT),
    (tensor(), mx(sr=64), None, INVALID), (tensor(), mx(sr=136), None, ALIGNMENT),
    (tensor(), mx(reserved=1), None, INVALID), (tensor(), mx(batch=0), None, INVALID),
    (tensor(batch=2), mx(batch=2, sb=64), None, INVALID), (tensor(batch=2), mx(batch=2, ss=256), None, INVALID),
    (tensor(batch=70000), mx(batch=70000), None, UNSUPPORTED),
    (tensor(), mx(), tensor(cols=120), INVALID), (tensor(), mx(), tensor(sr=100), INVALID),
    (tensor(), mx(), tensor(dtype=E4M3), UNSUPPORTED), (tensor(), mx(), tensor(sr=1, sc=64), UNSUPPORTED),
])
def test_quantize_refusals(lib, x, q, v, code):
    assert lib.gge_mx_quantize(ref(x), ref(q), ref(v), None) == code


def test_empty_calls_do_nothing(lib):
    x, q = tensor(0, 128, ptr=None), mx(0, 128, codes=None, scales=None)
    assert lib.gge_mx_quantize(ref(x), ref(q), None, None) == 0
    assert lib.gge_mx_dequantize(ref(q), ref(x), None) == 0
    args = b.GgeRmsnormArgs(x, None, None, None, None, None, P, BF16, 1e-5, None)
    assert lib.gge_rmsnorm(ref(args), None) == 0
    args = b.GgeRmsnormBwdArgs(x, x, None, x, P, BF16, 0, P, None)
    assert lib.gge_rmsnorm_bwd(ref(args), None, 0, None) == 0


@pytest.mark.parametrize("q,y,code", [
    (None, tensor(), INVALID), (mx(), None, INVALID), (mx(fmt=7), tensor(), INVALID),
    (mx(), tensor(rows=65), INVALID), (mx(), tensor(sr=64), INVALID), (mx(), tensor(sr=1, sc=64), UNSUPPORTED),
    (mx(), tensor(dtype=E4M3), UNSUPPORTED),
])
def test_dequantize_refusals(lib, q, y, code):
    assert lib.gge_mx_dequantize(ref(q), ref(y), None) == code


def product(lib, A=None, B=None, C=None, D=tensor(64, 72, sr=72), P_=None, act=0, config=None, ws=P, n=256,
            reserved=0, dact=False):
    A = A if A is not None else mx(64, 128)
    B = B if B is not None else mx(72, 128)
    args = b.GgeGemmMxArgs(A, B, ref(C), ref(D), ref(P_), 1.0, 0.0, None, None, act, reserved, ref(config))
    fn = lib.gge_gemm_mx_dact if dact else lib.gge_gemm_mx
    return fn(ref(args), ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=None), INVALID), (dict(act=9), INVALID), (dict(act=1), INVALID), (dict(reserved=1), INVALID),
    (dict(A=mx(64, 128, 1)), UNSUPPORTED), (dict(A=mx(63, 128)), INVALID), (dict(B=mx(72, 96)), INVALID),
    (dict(A=mx(64, 128, batch=2)), INVALID),
    (dict(B=mx(68, 128), D=tensor(64, 68, sr=72)), UNSUPPORTED),
    (dict(D=tensor(64, 72, sr=73)), ALIGNMENT), (dict(D=tensor(64, 72, sr=72, ptr=P + 8)), ALIGNMENT),
    (dict(D=tensor(64, 72, sr=64)), INVALID), (dict(D=tensor(64, 72, dtype=E4M3)), UNSUPPORTED),
    (dict(C=tensor(64, 80, sr=80)), INVALID), (dict(n=128), WORKSPACE), (dict(ws=P + 4), ALIGNMENT),
    (dict(config=b.make_config(tile_n=192)), UNSUPPORTED), (dict(config=b.make_config(stages=1)), UNSUPPORTED),
    (dict(config=b.make_config(flags=4)), UNSUPPORTED), (dict(config=b.make_config(cta_group=2)), UNSUPPORTED),
    (dict(dact=True, act=3), INVALID), (dict(dact=True, C=tensor(64, 72, sr=72)), INVALID),
    (dict(dact=True, C=tensor(64, 72, sr=72), act=3, D=None, P_=tensor(64, 72, sr=72)), INVALID),
])
def test_product_refusals(lib, kw, code):
    assert product(lib, **kw) == code


def test_null_arguments(lib):
    assert lib.gge_gemm_mx(None, P, 256, None) == INVALID
    assert lib.gge_gemm_mx_dact(None, P, 256, None) == INVALID
    assert lib.gge_rmsnorm(None, None) == INVALID
    assert lib.gge_rmsnorm_bwd(None, None, 0, None) == INVALID


def norm(lib, x=tensor(), residual=None, out=None, y=tensor(), q=None, values=None, weight=P, wt=BF16, inv=P):
    args = b.GgeRmsnormArgs(x, ref(residual), ref(out), ref(y), ref(q), ref(values), weight, wt, 1e-5, inv)
    return lib.gge_rmsnorm(ref(args), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=tensor(batch=2)), UNSUPPORTED), (dict(x=tensor(dtype=E4M3)), UNSUPPORTED),
    (dict(x=tensor(sr=1, sc=64)), UNSUPPORTED), (dict(weight=None), INVALID), (dict(wt=E4M3), UNSUPPORTED),
    (dict(weight=P + 1), ALIGNMENT), (dict(inv=P + 2), ALIGNMENT), (dict(y=tensor(dtype=F16)), UNSUPPORTED),
    (dict(y=tensor(rows=60)), INVALID), (dict(y=tensor(sr=100)), INVALID),
    (dict(residual=tensor(dtype=F32)), UNSUPPORTED), (dict(out=tensor()), INVALID),
    (dict(residual=tensor(), out=tensor(sr=100)), INVALID), (dict(values=tensor()), INVALID),
    (dict(q=mx(64, 96)), INVALID), (dict(q=mx(fmt=5)), INVALID), (dict(q=mx(), values=tensor(cols=96)), INVALID),
    (dict(q=mx(64, 128, batch=2)), INVALID),
])
def test_norm_refusals(lib, kw, code):
    assert norm(lib, **kw) == code


def norm_bwd(lib, dy=tensor(), h=tensor(), dh=None, dx=tensor(), weight=P, wt=BF16, inv=P, dw=None, reserved=0):
    args = b.GgeRmsnormBwdArgs(dy, h, ref(dh), dx, weight, wt, reserved, inv, dw)
    return lib.gge_rmsnorm_bwd(ref(args), None, 0, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dy=tensor(batch=2)), UNSUPPORTED), (dict(h=tensor(dtype=F16)), UNSUPPORTED),
    (dict(h=tensor(cols=64)), INVALID), (dict(dh=tensor(rows=3)), INVALID), (dict(dx=tensor(sr=100)), INVALID),
    (dict(weight=None), INVALID), (dict(inv=None), INVALID), (dict(inv=P + 1), ALIGNMENT),
    (dict(dw=P + 2), ALIGNMENT), (dict(wt=E4M3), UNSUPPORTED), (dict(reserved=1), INVALID),
])
def test_norm_bwd_refusals(lib, kw, code):
    assert norm_bwd(lib, **kw) == code


def test_workspace_size_without_a_gpu_or_with_one(lib):
    n = [lib.gge_workspace_size_rmsnorm_bwd(c) for c in (0, 1, 1000)]
    assert lib.gge_workspace_size_rmsnorm_bwd(-1) == 0
    assert n == [0, 0, 0] or (n[0] > 0 and n[2] - n[0] == 1000 * (n[1] - n[0]))


def batched(sb, sr=128, rows=64, cols=128, batch=3):
    return tensor(rows, cols, batch=batch, sr=sr, sb=sb)


OVERLAPPING = [batched(0), batched(64 * 128 - 128), batched(128), batched(128, sr=256), batched(0, rows=1)]
# (one row a batch; batches after one another; row r of every batch side by side)
APART = [batched(128, rows=1), batched(64 * 128), batched(128, sr=384)]


@pytest.mark.parametrize("v", OVERLAPPING)
def test_outputs_whose_batches_overlap_are_refused(lib, v):
    """(they would be written in no particular order)"""
    rows = v.rows
    q = mx(rows, 128, batch=3)
    x = tensor(rows, 128, batch=3)
    assert lib.gge_mx_quantize(ref(x), ref(q), ref(v), None) == INVALID
    assert lib.gge_mx_dequantize(ref(q), ref(v), None) == INVALID
    B = mx(128, 128, batch=3)
    for kw in (dict(D=v), dict(D=tensor(rows, 128, batch=3), P_=v, act=1)):
        assert product(lib, A=q, B=B, **kw) == INVALID
    assert product(lib, A=q, B=B, D=v, C=tensor(rows, 128, batch=3), act=3, dact=True) == INVALID


@pytest.mark.parametrize("v", APART)
def test_inputs_may_overlap_and_outputs_lie_apart_in_either_order(lib, v):
    """What these calls refuse instead comes after the outputs' check: the workspace."""
    q, B = mx(v.rows, 128, batch=3), mx(128, 128, batch=3)
    assert product(lib, A=q, B=B, D=v, C=tensor(v.rows, 128, batch=3, sb=0), n=128) == WORKSPACE


def test_transposed_source_of_too_many_rows_is_refused(lib):
    rows = 65535 * 64 + 1
    x = tensor(rows, 2, sr=1, sc=rows)
    assert lib.gge_mx_quantize(ref(x), ref(mx(rows, 2)), None, None) == UNSUPPORTED
