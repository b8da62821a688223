"""MxTensor and mx_empty as objects (host logic; the compiled module is stood in for)."""

import pytest
import torch

from grouped_gemm_epilogues_gb300 import binding as b

DEV = torch.device("cuda", 0)


class _Marshal:
    """mx_alloc over CPU memory, with the struct as the compiled module fills it."""

    def mx_alloc(self, nbytes, start, device, fmt, rows, cols, batch, row, per, scale):
        buf = torch.zeros(nbytes, dtype=torch.uint8)
        p = buf.data_ptr()
        c = b.GgeMxTensor(p, p + start, scale.data_ptr() if scale is not None else None, fmt, 0, rows, cols,
                          batch if batch > 0 else 1, row, rows * row if batch > 0 else 0, per)
        return buf, bytes(c)


@pytest.fixture(autouse=True)
def marshal(monkeypatch):
    monkeypatch.setattr(b, "_marshal", _Marshal())


def test_what_the_struct_holds_cannot_be_assigned():
    """The kernels read the struct made at construction: an assignment would do nothing."""
    t = torch.ones(1)
    q = b.mx_empty(4, 64, "nvfp4", device=DEV, tensor_scale=t)
    assert q.tensor_scale is t and q.format == "nvfp4" and q.device == DEV and (q.rows, q.cols, q.batch) == (4, 64, 1)
    for name, value in (("tensor_scale", torch.ones(1)), ("format", "mxfp4"), ("device", torch.device("cpu")),
                        ("rows", 3), ("codes", None), ("scales", None), ("c", b"")):
        with pytest.raises(AttributeError):
            setattr(q, name, value)
    assert q.tensor_scale is t


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
def test_mx_empty_shapes(fmt):
    """codes have a batch dimension exactly where one was asked for, however many rows."""
    row = b._mx_row_bytes(b.MX_FORMAT[fmt], 100)
    for rows in (0, 1, 130):
        per = b._mx_scale_bytes(b.MX_FORMAT[fmt], rows, 100)
        q = b.mx_empty(rows, 100, fmt, device=DEV)
        assert q.codes.shape == (rows, row) and q.scales.shape == (per,) and q.batch == 1
        for batch in (1, 3):
            q = b.mx_empty(rows, 100, fmt, device=DEV, batch=batch)
            assert q.codes.shape == (batch, rows, row) and q.scales.shape == (batch * per,) and q.batch == batch


@pytest.mark.parametrize("rows,cols,batch", [(4, 64, 0), (4, 64, -1), (-4, 64, None), (4, -64, None), (-4, -64, 2)])
def test_mx_empty_refuses_sizes_that_hold_nothing(rows, cols, batch):
    """(batch=0 came out as one batch without memory)"""
    with pytest.raises(ValueError, match="mx_empty"):
        b.mx_empty(rows, cols, "mxfp8", device=DEV, batch=batch)
