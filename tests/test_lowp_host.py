"""Host-side arithmetic and host code of the low-precision layer, compiled by itself and
run on the CPU."""

import os
import re
import subprocess

import torch

from grouped_gemm_epilogues_gb300 import binding as b, build

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


LIMIT = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include "gge_launch.h"
// a device whose blocks may have 232448 bytes, kernels with 256 and 1024 static ones, and
// attribute calls that take their time
static std::atomic<int> limit[3], sets;
void kern(int) {}
void other(int) {}
static int which(const void* f) { return f == reinterpret_cast<const void*>(kern) ? 0 : 1; }
static thread_local int device = 0;
extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t cudaThreadExchangeStreamCaptureMode(cudaStreamCaptureMode*) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrMaxSharedMemoryPerBlockOptin ? 232448 : -1;
  return cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void* f) {
  a->sharedSizeBytes = which(f) == 0 ? 256 : 1024;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute, int v) {
  std::this_thread::sleep_for(std::chrono::milliseconds(20 + 30 * (sets++ % 3)));
  limit[device == 0 ? which(f) : 2] = v;
  std::this_thread::sleep_for(std::chrono::milliseconds(20));
  return cudaSuccess;
}
}
int main() {
  std::atomic<int> short_of{0};
  std::thread t[8];
  for (int i = 0; i < 8; ++i)
    t[i] = std::thread([i, &short_of] {
      std::this_thread::sleep_for(std::chrono::milliseconds(7 * i));
      for (int n = 0; n < 5; ++n) {
        if (gge::allow_smem<kern>() != cudaSuccess || limit[0] != 232448 - 256) ++short_of;
        if (gge::allow_smem<other>() != cudaSuccess || limit[1] != 232448 - 1024) ++short_of;
      }
    });
  for (auto& x : t) x.join();
  const int before = sets;
  gge::allow_smem<kern>();
  const int again = sets - before;
  device = 1;
  gge::allow_smem<kern>();
  std::printf("%d %d %d\n", (int)short_of, again, (int)limit[2]);
}
"""


def test_shared_memory_limit_of_first_calls_in_several_threads(tmp_path):
    """Whatever the order of their calls, no thread finds a limit below the device's, and a
    kernel's limit is set on each device."""
    src, exe = tmp_path / "limit.cpp", tmp_path / "limit"
    src.write_text(LIMIT)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    r = subprocess.run(["g++", "-std=c++17", "-I", build.CSRC, "-I", cuda, str(src), "-o", str(exe), "-lpthread"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.stdout.split() == ["0", "0", str(232448 - 256)], r.stdout + r.stderr


def test_compiled_module_calls_the_library_with_the_tensors_device_current():
    """(A second device is what would show it; here, that the one macro does it for every call.)"""
    text = open(os.path.join(LOWP, "marshal.cpp")).read()
    macro = text[text.index("#define GGE_CALL"):]
    macro = macro[:macro.index("\n\n")]
    assert macro.index("CUDAGuard") < macro.index("stream(dev)") < macro.index("(expr)")
    host_only = {"gge_mx_row_bytes", "gge_mx_scale_bytes"}
    for name in re.findall(r"\b(gge_\w+)\(", text):
        if name in b._SIGNATURES and name not in host_only and name != "gge_workspace_size_rmsnorm_bwd":
            line = next(x for x in text.splitlines() if name + "(" in x and not x.startswith("//"))
            assert line.strip().startswith("GGE_CALL(dev, "), line
    at = text.index("gge_workspace_size_rmsnorm_bwd(")
    assert "CUDAGuard" in text[text.rindex("{", 0, at):at]
