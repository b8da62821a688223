"""Builds libgge.so in-tree with nvcc for sm_103a.

Each .cu under csrc/ and csrc/lowp/ is compiled in parallel into _build/, then linked into
``_build/libgge.so``.  ``python -m grouped_gemm_epilogues_gb300.build`` or
``build()`` from Python; ``-Xptxas -v`` output goes to ``_build/ptxas.log``.
csrc/lowp/marshal.cpp becomes ``_build/gge_marshal.<Python>-torch<version>.so``, a Python
module over libgge.so, where torch is installed; the library does not need it.
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
MARSHAL_SOURCE = os.path.join(CSRC, "lowp", "marshal.cpp")

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


def _headers():
    return (glob.glob(os.path.join(CSRC, "**", "*.cuh"), recursive=True) +
            glob.glob(os.path.join(CSRC, "**", "*.h"), recursive=True) +
            glob.glob(os.path.join(ROOT, "include", "*.h")))


def _lib_deps():
    return _sources() + _headers()


def _torch():
    try:
        import torch
    except ImportError:
        return None
    return torch


def marshal_path():
    """The Python module's file for this Python and torch (its binary interface is theirs), or
    None without torch."""
    torch = _torch()
    if torch is None:
        return None
    return os.path.join(BUILD, f"gge_marshal.{sysconfig.get_config_var('SOABI')}-torch{torch.__version__}.so")


def _compile(src: str) -> tuple:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc()] + ARCH + NVCC_FLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    return obj, r.returncode, r.stdout + r.stderr, " ".join(cmd)


def _gxx(cmd) -> None:
    try:
        r = subprocess.run(["g++"] + cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"gge_marshal: {e}") from e
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("gge_marshal: g++ " + " ".join(cmd))


def _compile_marshal(obj: str) -> None:
    """The Python module's object file (torch's and CPython's headers)."""
    torch = _torch()
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    _gxx(["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
          "-isystem", cuda, "-isystem", sysconfig.get_paths()["include"], "-c", MARSHAL_SOURCE, "-o", obj])


def _link_marshal(obj: str, path: str) -> None:
    lib = os.path.join(os.path.dirname(_torch().__file__), "lib")
    tmp = path + ".tmp"
    _gxx(["-shared", "-o", tmp, obj, "-L", BUILD, "-L", lib, "-lgge", "-ltorch_python",
          "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib])
    os.replace(tmp, path)


def _newer(path: str, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps)


def _lib_up_to_date() -> bool:
    return _newer(LIB, _lib_deps())


def _marshal_up_to_date() -> bool:
    path = marshal_path()
    return path is None or _newer(path, [MARSHAL_SOURCE] + _headers())


def up_to_date() -> bool:
    return _lib_up_to_date() and _marshal_up_to_date()


def _link(objects) -> None:
    tmp = LIB + ".tmp"
    # no -lcuda: the driver entry point (cuTensorMapEncodeTiled) is resolved at run time
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objects
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("link failed")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    path, marshal = marshal_path(), None
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        if path is not None and (force or not _marshal_up_to_date()):
            marshal = ex.submit(_compile_marshal, path[:-3] + ".o")
        results = list(ex.map(_compile, _sources())) if force or not _lib_up_to_date() else []
    if results:
        log = []
        for obj, rc, out, cmd in results:
            log.append(f"$ {cmd}\n{out}")
            if rc != 0:
                sys.stderr.write(out)
                raise RuntimeError(f"nvcc failed on {obj}")
        with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
            f.write("\n".join(log))
        _link([obj for obj, *_ in results])
        if verbose:
            print("\n".join(log))
    if marshal is not None:
        marshal.result()
        _link_marshal(path[:-3] + ".o", path)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
