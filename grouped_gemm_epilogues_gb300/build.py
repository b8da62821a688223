"""Builds libgge.so in-tree with nvcc for sm_103a.

Each .cu under csrc/ and csrc/lowp/ is compiled in parallel into _build/, then linked into
``_build/libgge.so``.  ``python -m grouped_gemm_epilogues_gb300.build`` or
``build()`` from Python; ``-Xptxas -v`` output goes to ``_build/ptxas.log``.
csrc/lowp/marshal.cpp becomes ``_build/gge_marshal.so``, a Python module over libgge.so.
"""

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(BUILD, "libgge.so")
MARSHAL = os.path.join(BUILD, "gge_marshal.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) +
                  glob.glob(os.path.join(CSRC, "lowp", "*.cu")))


def _deps():
    return _sources() + [os.path.join(CSRC, "lowp", "marshal.cpp")] + sorted(glob.glob(os.path.join(CSRC, "**", "*.cuh"), recursive=True) +
                               glob.glob(os.path.join(CSRC, "**", "*.h"), recursive=True) +
                               glob.glob(os.path.join(ROOT, "include", "*.h")))


def _compile(src: str) -> tuple:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc()] + ARCH + NVCC_FLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    return obj, r.returncode, r.stdout + r.stderr, " ".join(cmd)


def _compile_marshal(obj: str) -> tuple:
    """The Python module's object file (torch's and CPython's headers)."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", cuda, "-isystem", sysconfig.get_paths()["include"],
           "-c", os.path.join(CSRC, "lowp", "marshal.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    return obj, r.returncode, r.stdout + r.stderr, " ".join(cmd)


def _link_marshal(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = MARSHAL + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", BUILD, "-L", lib, "-lgge", "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("link of gge_marshal failed")
    os.replace(tmp, MARSHAL)


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MARSHAL):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(MARSHAL))
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        marshal_obj = os.path.join(BUILD, "marshal.o")
        marshal = ex.submit(_compile_marshal, marshal_obj)
        results = list(ex.map(_compile, _sources()))
        marshal = marshal.result()
    log = []
    for obj, rc, out, cmd in results + [marshal]:
        log.append(f"$ {cmd}\n{out}")
        if rc != 0:
            sys.stderr.write(out)
            raise RuntimeError(f"nvcc failed on {obj}")
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        f.write("\n".join(log))
    tmp = LIB + ".tmp"
    # no -lcuda: the driver entry point (cuTensorMapEncodeTiled) is resolved at run time
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + [o for o, *_ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("link failed")
    os.replace(tmp, LIB)
    _link_marshal(marshal_obj)
    if verbose:
        print("\n".join(log))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
