"""The shared workspace's life (host logic: the device's memory and the library are stood in
for): what a call replaces stays, because a captured graph may go on using it."""

import pytest
import torch

from grouped_gemm_epilogues_gb300 import binding as b

DEV = torch.device("cuda", 0)


class _Lib:
    """gge_read_device_status over CPU memory: the first word is the status, read and cleared."""

    def gge_read_device_status(self, ptr, stream, detail):
        for t in self.tensors:
            if t.data_ptr() == ptr.value:
                code = int(t[0])
                detail[0], detail[1] = int(t[1]), int(t[2])
                t[:16] = 0
                return code
        raise AssertionError("status of memory that is not a workspace")


@pytest.fixture
def lib(monkeypatch):
    lib = _Lib()
    lib.tensors = []

    def zeroed(dev, nbytes):
        assert dev == DEV
        lib.tensors.append(torch.zeros(nbytes, dtype=torch.uint8))
        return lib.tensors[-1]

    monkeypatch.setattr(b, "_workspaces", {})
    monkeypatch.setattr(b, "_replaced", {})
    monkeypatch.setattr(b, "_zeroed", zeroed)
    monkeypatch.setattr(b, "load", lambda: lib)
    monkeypatch.setattr(b, "_stream", lambda t: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: DEV.index)
    return lib


def test_replaced_workspaces_stay_alive(lib):
    first = b.workspace(DEV, 300)
    assert b.workspace(DEV, 300) is first and b.workspace(DEV) is first
    second = b.workspace(DEV, 1000)
    assert second is not first and second.numel() >= 1000
    assert any(t is first for t in b._replaced[0])
    # growth at least doubles, so what is kept is no more than what is in use
    for n in range(1000, 20000, 100):
        ws = b.workspace(DEV, n)
    assert sum(t.numel() for t in b._replaced[0]) <= ws.numel()


def test_status_of_a_replaced_workspace_is_read(lib):
    """A graph captured with it records its errors there."""
    first = b.workspace(DEV, 300)
    second = b.workspace(DEV, 1000)
    assert not second.any()
    assert b.gge_read_device_status(DEV)[0] == "GGE_OK"
    code = next(k for k, v in b.STATUS.items() if v == "GGE_ERR_TIMEOUT")
    first[0], first[1], first[2] = code, 3, 7
    assert b.gge_read_device_status(DEV) == ("GGE_ERR_TIMEOUT", 3, 7)
    assert b.gge_read_device_status(DEV)[0] == "GGE_OK"
    second[0], first[0] = code, code
    assert [b.gge_read_device_status(DEV)[0] for _ in range(3)] == ["GGE_ERR_TIMEOUT"] * 2 + ["GGE_OK"]
    own = torch.zeros(256, dtype=torch.uint8)
    lib.tensors.append(own)
    first[0] = code
    assert b.gge_read_device_status(workspace=own)[0] == "GGE_OK"
