"""8-bit outputs of 256-wide tiles without a C whose rows end on 16 codes leave by TMA, in boxes of 32
rows x 128 columns: alone, two of them, and beside 16- and 32-bit outputs whose chunks go through the
same buffers; boxes that end at N, at a batch's last row and inside a group; several tiles a CTA.
Codes and scales lie inside larger buffers whose other values have to stay.

Against the float64 oracle, within the tolerances of test_b128_gpu.py (derived there)."""

import numpy as np
import pytest
import torch

from grouped_gemm_epilogues_gb300 import binding as gge
from oracle import activations, formats, gemm as og

from helpers import FMT, dec
from test_b128_gpu import CODES, _check_q, _groups, _held, _numbers, _slack, _status, _x

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
KINDS = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CODE, SCALE, VALUE = 0xA5, 5.0, 77.0


class Output:
    """An output of one kind in the middle of larger buffers."""

    def __init__(self, kind, m, n, batch=None, interleaved=False):
        lead = batch or 1
        self.kind, self.m, self.n, self.batch = kind, m, n, batch

        def room(rows, cols, dtype, fill):
            """(batch, rows, cols) with a row or two around each batch and columns behind."""
            if interleaved and kind in KINDS:     # (codes take batches behind one another only)
                t = torch.full((rows + 3, lead, cols), fill, dtype=dtype, device=DEV)
                return t, t.transpose(0, 1)[:, 1:rows + 1]
            t = torch.full((lead, rows + 3, cols), fill, dtype=dtype, device=DEV)
            return t, t[:, 1:rows + 1]

        if kind in CODES:
            self.buffer, at = room(m, n + 48, torch.uint8, CODE)
            self.codes = at[:, :, 16:16 + n]
            self.scale_buffer, at = room((n + 127) // 128, m + 4, torch.float32, SCALE)
            self.scales = at[:, :, 2:2 + m].transpose(1, 2)
            codes = self.codes.view(CODES[kind])
            self.arg = gge.B128Tensor(codes, self.scales) if batch else gge.B128Tensor(codes[0], self.scales[0])
        else:
            self.buffer, at = room(m, n + 16, KINDS[kind], VALUE)
            self.value = at[:, :, 8:8 + n]
            self.arg = self.value if batch else self.value[0]

    def check(self, want, tol, rows=None):
        """The first `rows` rows against `want` (batch, m, n); whatever else the buffers hold is as it was."""
        rows = self.m if rows is None else rows
        if self.kind in CODES:
            for b in range(self.batch or 1):
                q = gge.B128Tensor(self.codes[b, :rows].view(CODES[self.kind]), self.scales[b, :rows])
                _check_q(q, want[b, :rows], tol[b, :rows])
            self.codes[:, :rows] = CODE
            self.scales[:, :rows] = SCALE
            assert (self.buffer == CODE).all() and (self.scale_buffer == SCALE).all()
        else:
            fmt = FMT[KINDS[self.kind]]
            r = formats.round_to(want[:, :rows], fmt)
            worst = np.abs(dec(self.value[:, :rows]) - r) / (tol[:, :rows] + formats.quantum(r, fmt))
            assert worst.max() <= 1.0, worst.max()
            self.value[:, :rows] = VALUE
            assert (self.buffer == VALUE).all()


PAIRS = [("e4m3", None), ("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "bf16"), ("f16", "e4m3"), ("e4m3", "f32"),
         ("f32", "e5m2"), (None, "e4m3")]


def _outputs(d, p, m, n, batch=None, interleaved=False):
    return [Output(kind, m, n, batch, interleaved) if kind else None for kind in (d, p)]


def _check_both(outs, act, ref, rows=None):
    v, bound = ref["v"], ref["bound"]
    if v.ndim == 2:
        v, bound = v[None], bound[None]
    if outs[0]:
        outs[0].check(v, _slack("none", v, bound), rows)
    if outs[1]:
        outs[1].check(activations.apply(act, v), _slack(act, v, bound), rows)


@pytest.mark.parametrize("d,p", PAIRS)
@pytest.mark.parametrize("m,n,k", [(256, 16, 130), (257, 80, 300), (2, 144, 260), (31, 272, 100), (700, 528, 140),
                                   (288, 1040, 64)])
@pytest.mark.parametrize("ctas", [0, 2])
def test_mixed_outputs(d, p, m, n, k, ctas):
    """ctas 2: one pair makes all tiles, so the next tile's outputs follow in the same buffers."""
    (A, av), (B, bv) = _held(_x(m, k, seed=m)), _held(_x(n, k, seed=n), 128)
    act = "gelu_tanh" if p else "none"
    ref = og.gemm(av[None], bv[None], alpha=0.5, act=act)
    outs = _outputs(d, p, m, n)
    gge.gge_gemm_b128(A, B, D=outs[0] and outs[0].arg, PostAct=outs[1] and outs[1].arg, act=act, alpha=0.5,
                      config=gge.make_config(tile_n=256, num_ctas=ctas))
    assert _status() == "GGE_OK"
    _check_both(outs, act, ref)


@pytest.mark.parametrize("d,p", PAIRS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("m,n,k", [(300, 144, 200), (40, 528, 130), (64, 16, 300)])
def test_batches(d, p, interleaved, m, n, k):
    batch = 3
    A, av = _held(torch.stack([_x(m, k, seed=s) for s in range(batch)]))
    B, bv = _held(torch.stack([_x(n, k, seed=10 + s) for s in range(batch)]), 128)
    act = "silu" if p else "none"
    ref = og.gemm(av, bv, act=act)
    for ctas in (0, 2):
        outs = _outputs(d, p, m, n, batch, interleaved)
        gge.gge_gemm_b128(A, B, D=outs[0] and outs[0].arg, PostAct=outs[1] and outs[1].arg, act=act,
                          config=gge.make_config(tile_n=256, num_ctas=ctas))
        assert _status() == "GGE_OK"
        _check_both(outs, act, ref)


@pytest.mark.parametrize("d,p", PAIRS)
@pytest.mark.parametrize("sizes", [[33, 0, 256, 1, 31, 64], [1] * 9, [0, 300, 0, 95], [32, 32, 96]])
@pytest.mark.parametrize("ctas", [0, 2])
def test_groups_that_end_inside_a_box(d, p, sizes, ctas):
    """Whole boxes and a group's last rows take turns in the same buffers; five rows lie behind
    the last group."""
    total, n, k = sum(sizes), 272, 200
    A, av = _held(_x(total + 5, k, seed=total))
    B, bv = _held(torch.stack([_x(n, k, seed=30 + g) for g in range(len(sizes))]), 128)
    cu = _groups(sizes)
    act = "gelu_tanh" if p else "none"
    ref = og.gemm_varlen_m(av, bv, cu.cpu().numpy())
    outs = _outputs(d, p, total + 5, n)
    gge.gge_gemm_b128_varlen_m(A, B, cu, D=outs[0] and outs[0].arg, PostAct=outs[1] and outs[1].arg, act=act,
                               config=gge.make_config(tile_n=256, num_ctas=ctas))
    assert _status() == "GGE_OK"
    _check_both(outs, act, ref, total)


@pytest.mark.parametrize("d,p,act", [("e4m3", "e4m3", "gelu_tanh"), ("bf16", "e4m3", "silu"), ("e4m3", None, "none"),
                                     ("bf16", "bf16", "gelu_tanh")])
def test_calls_repeat_bit_for_bit(d, p, act):
    """Several rounds of tiles on every pair, over and over: the same bits each time."""
    m, n, k = 2600, 2064, 520
    A, B = _held(_x(m, k))[0], _held(_x(n, k, seed=1), 128)[0]
    first = None
    for _ in range(20):
        outs = _outputs(d, p, m, n)
        gge.gge_gemm_b128(A, B, D=outs[0].arg, PostAct=outs[1] and outs[1].arg, act=act,
                          config=gge.make_config(tile_n=256, num_ctas=40))
        bits = [t for o in outs if o for t in ((o.codes, o.scales) if o.kind in CODES else (o.value.view(torch.int16),))]
        if first is None:
            first = [t.clone() for t in bits]
        assert all(torch.equal(a, b) for a, b in zip(bits, first))
    assert _status() == "GGE_OK"


def test_numbers_are_those_that_the_codes_stand_for():
    """(the checks above read codes on the host: the device's decoding agrees)"""
    A, B = _held(_x(300, 200))[0], _held(_x(144, 200, seed=1), 128)[0]
    out = Output("e4m3", 300, 144)
    gge.gge_gemm_b128(A, B, D=out.arg, config=gge.make_config(tile_n=256))
    y = torch.empty(300, 144, device=DEV)
    gge.gge_b128_dequantize(out.arg, y)
    assert np.array_equal(dec(y), formats.round_to(_numbers(out.arg), formats.F32))
