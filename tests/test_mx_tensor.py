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
