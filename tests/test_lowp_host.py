"""Host-side arithmetic and host code of the low-precision layer, compiled by itself and
run on the CPU."""

import os
import subprocess

import torch

from grouped_gemm_epilogues_gb300 import build

LOWP = os.path.join(build.CSRC, "lowp")


def _run(tmp_path, source, *args):
    """Compile a program with nvcc (host code only: no device is touched) and run it."""
    src, exe = tmp_path / "prog.cu", tmp_path / "prog"
    src.write_text(source)
    r = subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-I", build.CSRC, "-I", LOWP, str(src), "-o",
                        str(exe), *args], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


SPAN = r"""
#include <cstdio>
#include "mx_format.cuh"
int main() {
  using namespace gge::mx;
  long long kg;
  for (long long k : {0LL, 1LL, 129LL, (1LL << 23) + 1, (1LL << 24) - 1, 1LL << 24, (1LL << 24) + 1, (1LL << 25) - 65}) {
    kg = k;
    std::printf("%lld %lld %lld %lld\n", kg, (long long)scale_span<FMT_MXFP8>(kg),
                (long long)scale_span<FMT_MXFP4>(kg), (long long)scale_span<FMT_NVFP4>(kg));
  }
}
"""


def test_scale_span_in_64_bits_and_by_the_format_s_group(tmp_path):
    """A scale word covers four blocks: 128 columns, nvfp4 64.  A row may have 2^31 - 4097
    columns, nearly 2^25 words of nvfp4."""
    rows = [tuple(map(int, line.split())) for line in _run(tmp_path, SPAN).splitlines()]
    assert len(rows) == 8
    for kg, mxfp8, mxfp4, nvfp4 in rows:
        assert (mxfp8, mxfp4, nvfp4) == (128 * kg, 128 * kg, 64 * kg)


class _Marshal:
    """Stands in for the compiled module: keeps each call's arguments, reports success."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


def test_backward_norm_does_not_keep_its_partial_sums_in_the_shared_workspace(monkeypatch):
    """They grow with the width: a captured graph would go on writing to a workspace that a
    wider call has replaced.  The compiled module takes a buffer of the call's own."""
    from grouped_gemm_epilogues_gb300 import binding as b

    def refuse(*args):
        raise AssertionError("shared workspace")

    fake = _Marshal()
    monkeypatch.setattr(b, "_marshal", fake)
    monkeypatch.setattr(b, "_shared_workspace", refuse)
    monkeypatch.setattr(b, "load", refuse)
    x, v, row = torch.zeros(4, 8), torch.zeros(8), torch.zeros(4)
    b.gge_rmsnorm_bwd(x, x, v, row, x, dW=v)
    b.gge_rmsnorm_bwd(x, x, v, row, x)
    own = torch.zeros(1 << 20, dtype=torch.uint8)
    b.gge_rmsnorm_bwd(x, x, v, row, x, dW=v, workspace=own)
    assert [args[7] for _, args in fake.calls] == [None, None, own]
