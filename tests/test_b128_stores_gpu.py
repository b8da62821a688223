"""Outputs of 256-wide tiles without a C: 16-bit ones leave by TMA in boxes of 32 rows x 32 columns,
others and a group's last rows by the warps themselves, through the same buffers.  Every mix of them, at
sizes that end inside a box, against the same product in 128-wide tiles; what lies around an
output keeps its values.

Both sums are those of the same blocks in the same order, so before they are rounded they differ by a few
units of fp32 at most; rounded, by one step of the output's type: eps relative to the value, and
where an 8-bit scale or value may round the other way, two steps of the code (2 * 2^-3 of the value)."""

import pytest
import torch

from grouped_gemm_epilogues_gb300 import binding as gge

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
KINDS = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GUARD = 77.0


def held(rows, cols, block, batch=None, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + rows + cols)
    q = gge.b128_empty(rows, cols, block, device=DEV, batch=batch)
    x = torch.randn(*((batch,) if batch else ()), rows, cols, generator=g, device=DEV)
    gge.gge_b128_quantize(x, q)
    return q


class Output:
    """An output of one kind inside a larger buffer that holds GUARD elsewhere."""

    def __init__(self, kind, m, n, batch=None, side_by_side=False):
        self.kind = kind
        if kind == "8":
            self.arg = gge.b128_empty(m, n, device=DEV, batch=batch)
            return
        lead = (batch,) if batch else ()
        if side_by_side:     # batches interleaved row by row
            self.buffer = torch.full((m + 2, batch, n + 8), GUARD, dtype=KINDS[kind], device=DEV)
            self.arg = self.buffer[1:m + 1].transpose(0, 1)[:, :, :n]
        else:
            self.buffer = torch.full((*lead, m + 2, n + 8), GUARD, dtype=KINDS[kind], device=DEV)
            self.arg = self.buffer[..., 1:m + 1, :n]

    def numbers(self, m, n, batch=None):
        if self.kind != "8":
            return self.arg.float()
        y = torch.empty(*((batch,) if batch else ()), m, n, device=DEV)
        gge.gge_b128_dequantize(self.arg, y)
        return y

    def guards_hold(self):
        if self.kind == "8":
            return True
        rest = self.buffer.clone()
        torch.as_strided(rest, self.arg.shape, self.arg.stride(), self.arg.storage_offset()).fill_(GUARD)
        return bool((rest == GUARD).all())


def check(a, b, kind):
    eps = 0.25 if kind == "8" else torch.finfo(KINDS[kind]).eps
    top = b.abs().amax(-1, keepdim=True) if kind == "8" else b.abs()
    # (a subnormal code's step is 2^-9 of the scale, which is 1 / 448 of the block's largest value; the
    # row's is at least that)
    slack = eps * b.abs() + (top * 2 ** -8 if kind == "8" else 4e-6 * b.abs().amax())
    assert bool(((a - b).abs() <= slack).all()), float(((a - b).abs() - slack).max())


@pytest.mark.parametrize("d,p", [("bf16", None), ("f16", "bf16"), (None, "f16"), ("f32", "bf16"), ("bf16", "f32"), ("8", "bf16"),
                                 ("f16", "8"), (None, "f32"), ("8", "8")])
@pytest.mark.parametrize("m,n,k", [(256, 8, 130), (257, 264, 300), (31, 40, 100), (700, 616, 140), (2, 72, 260)])
def test_mixed_outputs(d, p, m, n, k):
    A, B = held(m, k, 1), held(n, k, 128)
    got = []
    for tile in (256, 128):
        outs = [Output(kind, m, n) if kind else None for kind in (d, p)]
        gge.gge_gemm_b128(A, B, D=outs[0].arg if d else None, PostAct=outs[1].arg if p else None,
                          act="silu" if p else "none", alpha=0.5, config=gge.make_config(tile_n=tile, flags=32))
        got.append(outs)
    assert gge.gge_read_device_status(DEV)[0] == "GGE_OK"
    for wide, narrow, kind in zip(*got, (d, p)):
        if kind:
            assert wide.guards_hold() and narrow.guards_hold()
            check(wide.numbers(m, n), narrow.numbers(m, n), kind)


@pytest.mark.parametrize("side_by_side", [False, True])
@pytest.mark.parametrize("batch,m,n,k", [(3, 300, 136, 200), (2, 40, 520, 130)])
def test_batches_behind_one_another_or_interleaved(side_by_side, batch, m, n, k):
    A, B = held(m, k, 1, batch), held(n, k, 1, batch)
    outs = []
    for tile in (256, 128):
        o = Output("bf16", m, n, batch, side_by_side)
        gge.gge_gemm_b128(A, B, D=o.arg, config=gge.make_config(tile_n=tile, flags=32))
        assert o.guards_hold()
        outs.append(o.numbers(m, n))
    check(*outs, "bf16")


@pytest.mark.parametrize("sizes", [[33, 0, 256, 1, 31, 64], [1] * 9, [0, 300, 0, 95]])
@pytest.mark.parametrize("d,p", [("bf16", None), ("bf16", "f16"), (None, "8"), ("f32", "f16")])
def test_groups_end_inside_boxes_and_rows_behind_them_stay(sizes, d, p):
    total = sum(sizes) + 5          # (five rows behind the last group)
    n, k = 264, 200
    A, B = held(total, k, 1), held(n, k, 128, len(sizes))
    cu = torch.tensor([sum(sizes[:i]) for i in range(len(sizes) + 1)], dtype=torch.int32, device=DEV)
    got = []
    for tile in (256, 128):
        outs = [Output(kind, total, n) if kind else None for kind in (d, p)]
        gge.gge_gemm_b128_varlen_m(A, B, cu, D=outs[0].arg if d else None, PostAct=outs[1].arg if p else None,
                                   act="gelu_tanh" if p else "none", config=gge.make_config(tile_n=tile))
        got.append(outs)
    for wide, narrow, kind in zip(*got, (d, p)):
        if kind:
            assert wide.guards_hold() and narrow.guards_hold()
            if kind != "8":
                assert bool((wide.arg[-5:] == GUARD).all())
            check(wide.numbers(total, n)[:-5], narrow.numbers(total, n)[:-5], kind)
