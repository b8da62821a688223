"""Calls on tensors of a device that is not the current one (host logic; devices stood in for):
the library plans and launches on the current device, so the tensors' is made current."""

import contextlib

import pytest
import torch

from grouped_gemm_epilogues_gb300 import binding as b


class _Tensor:
    def __init__(self, device):
        self.device = torch.device(device)


class _Reached(Exception):
    pass


@pytest.fixture
def current(monkeypatch):
    """The current device's index, and what it was each time the library was reached."""
    state = {"now": 0, "seen": []}

    @contextlib.contextmanager
    def device(d):
        before, state["now"] = state["now"], torch.device(d).index
        try:
            yield
        finally:
            state["now"] = before

    @contextlib.contextmanager
    def reached():
        try:
            yield
        except _Reached:
            pass

    def load():
        state["seen"].append(state["now"])
        raise _Reached

    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["now"])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(b, "load", load)
    state["reached"] = reached
    return state


CALLS = {
    "gge_gemm": lambda t: b.gge_gemm(t, t, t),
    "gge_gemm_act": lambda t: b.gge_gemm_act(t, t, t, "relu"),
    "gge_gemm_dact": lambda t: b.gge_gemm_dact(t, t, t, t, "relu"),
    "gge_gemm_act_static_scratch": lambda t: b.gge_gemm_act_static_scratch(t, t, t, "relu"),
    "gge_gemm_varlen_m": lambda t: b.gge_gemm_varlen_m(t, t, t, D=t),
    "gge_gemm_varlen_k": lambda t: b.gge_gemm_varlen_k(t, t, t, D=t),
    "gge_gemm_gather_k": lambda t: b.gge_gemm_gather_k(t, t, t, t, D=t),
    "gge_gemm_gather_a": lambda t: b.gge_gemm_gather_a(A_src=t, B=t, a_idx=t, D=t),
    "gge_plan": lambda t: b.gge_plan(t, t, D=t),
    "gge_tune_candidates": lambda t: b.gge_tune_candidates("gemm", t, t, D=t),
    "gge_autotune": lambda t: b.gge_autotune("gemm", A=t, B=t, D=t),
    "gge_tuned_config": lambda t: b.gge_tuned_config("gemm", t, t, D=t),
    "gge_read_static_scratch_status": lambda t: b.gge_read_static_scratch_status(t.device),
    "gge_read_device_status": lambda t: b.gge_read_device_status(t.device),
}


@pytest.mark.parametrize("name", CALLS)
def test_the_tensors_device_is_current_inside_the_call(current, name):
    for device, want in (("cuda:1", 1), ("cuda:0", 0), ("cuda:2", 2), ("cpu", 0)):
        if device == "cpu" and "status" in name:
            continue
        with current["reached"]():
            CALLS[name](_Tensor(device))
        assert current["seen"][-1] == want and current["now"] == 0
    assert len(current["seen"]) >= 3
