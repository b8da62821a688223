"""A launch shape's first call on a device, captured into a CUDA graph.

The first call of a launch shape makes one-time device queries (the kernel's
shared-memory limit, its occupancy, the tensor-map encoder's entry point).
CUDA refuses such calls while the thread captures a stream in the default
(global) mode; the library makes them in relaxed mode, so the capture succeeds.
The call runs in a fresh process (nothing cached yet), its graph is replayed,
and the outputs are compared with the oracle here.
"""

import os
import subprocess
import sys

import pytest
import torch

from grouped_gemm_epilogues_gb300 import workloads as wl

from test_gemm_gpu import _check_plain

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys, torch
sys.path.insert(0, sys.argv[1])
from grouped_gemm_epilogues_gb300 import binding, workloads as wl
cg, out_path = int(sys.argv[2]), sys.argv[3]
w = wl.small("gemm_act_4096_bf16_gelu", 300, 520, 200, 2)
t = {k: v.cuda() for k, v in wl.make(w).items() if isinstance(v, torch.Tensor)}
D = torch.full((2, 300, 520), float("nan"), dtype=torch.bfloat16, device="cuda")
P = torch.full_like(D, float("nan"))
binding.workspace(torch.device("cuda", 0), 64 << 20)   # made (and zeroed) before the capture
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    binding.gge_gemm_act(t["A"], t["B"], P, w.act, D=D, C=t["C"], alpha=w.alpha, beta=w.beta,
                         config=binding.make_config(cta_group=cg, tile_n=256))
assert torch.isnan(D.float()).all(), "the captured call ran during the capture"
g.replay()
torch.cuda.synchronize()
assert binding.gge_read_device_status()[0] == "GGE_OK"
torch.save({"D": D.cpu(), "P": P.cpu()}, out_path)
"""


@pytest.mark.parametrize("cta_group", [1, 2])
def test_first_call_inside_graph_capture(tmp_path, cta_group):
    out_path = str(tmp_path / "out.pt")
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, str(cta_group), out_path],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    got = torch.load(out_path)
    w = wl.small("gemm_act_4096_bf16_gelu", 300, 520, 200, 2)
    _check_plain(w, wl.make(w), got)


EAGER_BETWEEN = r"""
import sys, torch
sys.path.insert(0, sys.argv[1])
from grouped_gemm_epilogues_gb300 import binding as b
dev = torch.device("cuda", 0)
g = torch.Generator(device=dev).manual_seed(1)
m, n, k = 4096, 4096, 4096       # (its last wave is split: tickets and partial sums in the workspace)
A, B = (torch.randn(r, k, generator=g, device=dev).bfloat16() for r in (m, n))
junk = [torch.full((1 << 22,), 0x01010101, dtype=torch.int32, device=dev) for _ in range(4)]
del junk                          # what a workspace that nobody zeroes may start with
D = [torch.empty(m, n, dtype=torch.bfloat16, device=dev) for _ in range(3)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    b.gge_gemm(A, B, D[0])
small = b.workspace(dev)
assert not small.any(), "the workspace is zeroed when the capture is over"
b.gge_gemm(A, B, D[1])            # on the same workspace, before the first replay
wide = b.workspace(dev, 2 * small.numel())
b.gge_gemm(A, B, D[2])
graph.replay()
graph.replay()
torch.cuda.synchronize()
assert b.gge_read_device_status(dev)[0] == "GGE_OK"
assert b.workspace(dev) is wide and any(t is small for t in b._replaced[0])
assert torch.equal(D[0], D[1]) and torch.equal(D[0], D[2])
want = A.float() @ B.float().t()
assert float((D[0].float() - want).norm() / want.norm()) < 2.0 ** -7
"""


def test_workspace_first_made_inside_a_capture():
    """Made beside the capture and zeroed at once, so that calls before the first replay can
    use it; the graph keeps its own when a longer one replaces it."""
    r = subprocess.run([sys.executable, "-c", EAGER_BETWEEN, ROOT], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]


THREADS = r"""
import sys, threading, torch
sys.path.insert(0, sys.argv[1])
from grouped_gemm_epilogues_gb300 import binding as b
dev = torch.device("cuda", 0)
g = torch.Generator(device=dev).manual_seed(1)
def draw(*shape):
    return torch.randn(*shape, generator=g, device=dev).bfloat16()
b.workspace(dev)
norms = [(draw(500, c), draw(c)) for c in (64, 512, 2048, 4096, 8192, 16384, 1003, 7999)]
wide = [draw(n, 1024) for n in (64, 128, 256, 512)]
qs = [b.mx_empty(w.shape[0], 1024, "mxfp8", device=dev) for w in wide]
torch.cuda.synchronize()
go, errors, outs = threading.Barrier(12), [], {}
def norm(i):
    x, w = norms[i]
    y = torch.empty_like(x)
    go.wait()
    b.gge_rmsnorm(x, w, Y=y)
    outs[i] = y
def product(i):
    d = torch.empty(wide[i].shape[0], wide[i].shape[0], dtype=torch.bfloat16, device=dev)
    go.wait()
    b.gge_mx_quantize(wide[i], qs[i])
    b.gge_gemm_mx(qs[i], qs[i], D=d, config=b.make_config(stages=2 + i))
def run(f, i):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            f(i)
            torch.cuda.current_stream().synchronize()
    except Exception as e:
        errors.append((f.__name__, i, repr(e)))
threads = [threading.Thread(target=run, args=(f, i)) for f, n in ((norm, 8), (product, 4)) for i in range(n)]
for t in threads: t.start()
for t in threads: t.join()
for i in range(8):          # and every shape still launches afterwards
    y = torch.empty_like(norms[i][0])
    b.gge_rmsnorm(*norms[i], Y=y)
    if not torch.equal(y, outs[i]): errors.append(("again", i))
torch.cuda.synchronize()
assert not errors, errors
assert b.gge_read_device_status(dev)[0] == "GGE_OK"
"""


def test_first_calls_in_several_threads():
    r = subprocess.run([sys.executable, "-c", THREADS, ROOT], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
