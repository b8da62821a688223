"""The build's two parts: the C library needs nvcc alone; the Python module over it needs
torch's headers and g++, and belongs to one torch and one Python."""

import os
import subprocess

import pytest
import torch

from grouped_gemm_epilogues_gb300 import build as b


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A library of one empty function, built in a folder of its own."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "out"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "out" / "libgge.so"))
    monkeypatch.setattr(b, "_sources", lambda: [str(src)])
    monkeypatch.setattr(b, "_lib_deps", lambda: [str(src)])
    return tmp_path


def test_library_is_linked_when_the_module_does_not_compile(small, monkeypatch):
    real = subprocess.run

    def run(cmd, *args, **kw):
        if cmd[0] == "g++":
            raise FileNotFoundError("g++")
        return real(cmd, *args, **kw)

    monkeypatch.setattr(b.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="gge_marshal"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.marshal_path())


def test_library_alone_without_torch(small, monkeypatch):
    monkeypatch.setattr(b, "_torch", lambda: None)
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert b.marshal_path() is None and b.up_to_date()


def test_module_of_another_torch_is_not_taken(small, monkeypatch):
    """It carries torch's and Python's version in its name, and alone is made again."""
    made = []
    monkeypatch.setattr(b, "_compile_marshal", lambda obj: None)
    monkeypatch.setattr(b, "_link_marshal", lambda obj, path: made.append(path) or open(path, "w").close())
    b.build()
    assert made == [b.marshal_path()] and b.up_to_date()
    assert torch.__version__ in made[0] and "cpython" in made[0]
    t = os.path.getmtime(b.LIB)
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert not b.up_to_date()
    b.build()
    assert len(made) == 2 and made[1] != made[0] and os.path.getmtime(b.LIB) == t
    b.build()
    assert len(made) == 2
