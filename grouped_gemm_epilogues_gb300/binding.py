"""Thin ctypes binding of libgge.so (include/gge.h).

Argument marshalling only: torch tensors are turned into the C structs
(device pointer, dtype code, extents, element strides) and handed to the C
entry points of the same names; every step of the computation runs in the
library's CUDA kernels.  PyTorch supplies device memory and the current
stream.  There is no fallback: if the library cannot be loaded, ``load()``
raises.
"""

import contextlib
import ctypes
import functools
import importlib.util
import inspect
import operator
import os
import threading

import torch

from . import build as _build

c_i32, c_i64, c_u32, c_u64 = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_uint64

DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2, torch.float8_e5m2: 3,
         torch.float32: 4}
ACT = {"none": 0, None: 0, "relu": 1, "gelu_tanh": 2, "gelu_tanh_approx": 2, "silu": 3,
       "relu_sq": 4}
STATUS = {0: "GGE_OK", 1: "GGE_ERR_INVALID_ARG", 2: "GGE_ERR_UNSUPPORTED",
          3: "GGE_ERR_ALIGNMENT", 4: "GGE_ERR_WORKSPACE", 5: "GGE_ERR_CUDA",
          6: "GGE_ERR_TIMEOUT", 7: "GGE_ERR_INDEX_RANGE"}


class GgeTensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", c_i32), ("reserved", c_i32),
                ("rows", c_i64), ("cols", c_i64), ("batch", c_i64),
                ("stride_row", c_i64), ("stride_col", c_i64), ("stride_batch", c_i64)]


class GgeConfig(ctypes.Structure):
    _fields_ = [("tile_n", c_i32), ("num_ctas", c_i32), ("raster_band", c_i32),
                ("stages", c_i32), ("flags", c_i32), ("cta_group", c_i32),
                ("tile_counts", ctypes.c_void_p), ("timeout_ns", c_u64),
                ("batch_idx_permute", ctypes.c_void_p)]


class GgeGemmArgs(ctypes.Structure):
    _fields_ = [("A", GgeTensor), ("B", GgeTensor),
                ("C", ctypes.POINTER(GgeTensor)), ("D", ctypes.POINTER(GgeTensor)),
                ("PostAct", ctypes.POINTER(GgeTensor)),
                ("alpha", ctypes.c_float), ("beta", ctypes.c_float),
                ("alpha_dev", ctypes.c_void_p), ("beta_dev", ctypes.c_void_p),
                ("act", c_i32), ("reserved", c_i32), ("config", ctypes.POINTER(GgeConfig))]


class GgePlanInfo(ctypes.Structure):
    _fields_ = [("tile_m", c_i32), ("tile_n", c_i32), ("tile_k", c_i32), ("stages", c_i32),
                ("num_tiles", c_i32), ("grid", c_i32), ("threads", c_i32),
                ("smem_bytes", c_i32), ("raster_band", c_i32), ("cta_group", c_i32),
                ("raster_along_n", c_i32), ("tail_tiles", c_i32), ("tail_splits", c_i32)]


class GgeMxTensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("tensor_scale", ctypes.c_void_p), ("format", c_i32), ("reserved", c_i32),
                ("rows", c_i64), ("cols", c_i64), ("batch", c_i64), ("stride_row", c_i64),
                ("stride_batch", c_i64), ("scale_stride_batch", c_i64)]


class GgeGemmMxArgs(ctypes.Structure):
    _fields_ = [("A", GgeMxTensor), ("B", GgeMxTensor), ("C", ctypes.c_void_p),
                ("D", ctypes.c_void_p), ("PostAct", ctypes.c_void_p),
                ("alpha", ctypes.c_float), ("beta", ctypes.c_float),
                ("alpha_dev", ctypes.c_void_p), ("beta_dev", ctypes.c_void_p),
                ("act", c_i32), ("reserved", c_i32), ("config", ctypes.c_void_p)]


class GgeRmsnormArgs(ctypes.Structure):
    _fields_ = [("x", GgeTensor), ("residual", ctypes.c_void_p),
                ("residual_out", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("q", ctypes.c_void_p), ("values", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("weight_dtype", c_i32), ("eps", ctypes.c_float), ("inv_rms", ctypes.c_void_p)]


class GgeRmsnormBwdArgs(ctypes.Structure):
    _fields_ = [("dy", GgeTensor), ("h", GgeTensor), ("dh", ctypes.c_void_p), ("dx", GgeTensor),
                ("weight", ctypes.c_void_p), ("weight_dtype", c_i32), ("reserved", c_i32),
                ("inv_rms", ctypes.c_void_p), ("dweight", ctypes.c_void_p)]


# every function include/gge.h declares, with its ctypes signature
_SIGNATURES = {
    "gge_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(GgeGemmArgs), c_i32]),
    "gge_workspace_size_varlen_k": (ctypes.c_size_t, [ctypes.POINTER(GgeGemmArgs), c_i32]),
    "gge_gemm": (c_i32, [ctypes.POINTER(GgeGemmArgs), ctypes.c_void_p, ctypes.c_size_t,
                         ctypes.c_void_p]),
    "gge_gemm_act": (c_i32, [ctypes.POINTER(GgeGemmArgs), ctypes.c_void_p, ctypes.c_size_t,
                             ctypes.c_void_p]),
    "gge_gemm_varlen_m": (c_i32, [ctypes.POINTER(GgeGemmArgs), ctypes.c_void_p, c_i32,
                                  ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "gge_gemm_varlen_k": (c_i32, [ctypes.POINTER(GgeGemmArgs), ctypes.c_void_p, c_i32,
                                  ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "gge_gemm_gather_k": (c_i32, [ctypes.POINTER(GgeGemmArgs), ctypes.c_void_p, ctypes.c_void_p,
                                  c_i32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "gge_gemm_gather_a": (c_i32, [ctypes.POINTER(GgeGemmArgs), ctypes.c_void_p, ctypes.c_void_p,
                                  c_i32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "gge_gemm_dact": (c_i32, [ctypes.POINTER(GgeGemmArgs), ctypes.c_void_p, ctypes.c_size_t,
                              ctypes.c_void_p]),
    "gge_gemm_act_static_scratch": (c_i32, [ctypes.POINTER(GgeGemmArgs), ctypes.c_void_p]),
    "gge_read_device_status": (c_i32, [ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.POINTER(c_i32)]),
    "gge_read_static_scratch_status": (c_i32, [ctypes.c_void_p, ctypes.POINTER(c_i32)]),
    "gge_status_string": (ctypes.c_char_p, [c_i32]),
    "gge_fastdivmod_params": (None, [c_i32, ctypes.POINTER(c_u32), ctypes.POINTER(c_u32)]),
    "gge_fastdivmod_div": (c_i32, [c_i32, c_i32]),
    "gge_schedule_map": (c_i32, [c_i32, c_i32, c_i32, c_i32, c_i32, c_i32,
                                 ctypes.POINTER(c_i32)]),
    "gge_plan": (c_i32, [ctypes.POINTER(GgeGemmArgs), c_i32, c_i32, ctypes.POINTER(GgePlanInfo)]),
    "gge_version": (ctypes.c_char_p, []),
    "gge_tune_candidates": (c_i32, [ctypes.POINTER(GgeGemmArgs), c_i32, c_i32,
                                    ctypes.POINTER(GgeConfig), c_i32]),
    "gge_autotune": (c_i32, [ctypes.POINTER(GgeGemmArgs), c_i32, ctypes.c_void_p, ctypes.c_void_p,
                             c_i32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, c_i32,
                             ctypes.POINTER(GgeConfig), ctypes.POINTER(ctypes.c_float)]),
    "gge_tuned_config": (c_i32, [ctypes.POINTER(GgeGemmArgs), c_i32, c_i32,
                                 ctypes.POINTER(GgeConfig)]),
    "gge_mx_row_bytes": (ctypes.c_size_t, [c_i32, c_i64]),
    "gge_mx_scale_bytes": (ctypes.c_size_t, [c_i32, c_i64, c_i64]),
    "gge_mx_quantize": (c_i32, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                ctypes.c_void_p]),
    "gge_mx_dequantize": (c_i32, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "gge_gemm_mx": (c_i32, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "gge_gemm_mx_dact": (c_i32, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                 ctypes.c_void_p]),
    "gge_rmsnorm": (c_i32, [ctypes.c_void_p, ctypes.c_void_p]),
    "gge_workspace_size_rmsnorm_bwd": (ctypes.c_size_t, [c_i64]),
    "gge_rmsnorm_bwd": (c_i32, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                ctypes.c_void_p]),
}

_lib = None
_marshal = None
_lock = threading.Lock()


class GgeError(RuntimeError):
    def __init__(self, code, where=""):
        self.code = code
        self.name = STATUS.get(code, str(code))
        super().__init__(f"{where}: {self.name}")


def load(path: str = None, build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libgge.so (building it in-tree first if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = path or _build.LIB
        if not os.path.exists(path):
            if not build_if_missing:
                raise FileNotFoundError(path)
            _build.build()
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _load_marshal():
    """The compiled marshalling of the low-precision entry points (gge_marshal)."""
    global _marshal
    load()
    with _lock:
        if _marshal is None:
            path = _build.marshal_path()
            if not os.path.exists(path):
                _build.build()
            spec = importlib.util.spec_from_file_location("gge_marshal", path)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            _marshal = module
    return _marshal


# ---------------------------------------------------------------- marshalling

def view(t: torch.Tensor, kind: str) -> GgeTensor:
    """C view of a torch tensor.  kind: 'mk' (A), 'nk' (B) or 'mn' (C/D/PostAct);
    2-D tensors are one batch, 3-D tensors are (batch, rows, cols)."""
    if t.dim() == 2:
        rows, cols = t.shape
        batch, sr, sc, sb = 1, t.stride(0), t.stride(1), t.numel()
    elif t.dim() == 3:
        batch, rows, cols = t.shape
        sb, sr, sc = t.stride()
    else:
        raise ValueError(f"{kind}: expected a 2-D or 3-D tensor")
    if t.dtype not in DTYPE:
        raise TypeError(f"{kind}: unsupported dtype {t.dtype}")
    return GgeTensor(ctypes.c_void_p(t.data_ptr()), DTYPE[t.dtype], 0, rows, cols, batch,
                     sr, sc, sb)


_workspaces = {}   # per device index
_replaced = {}     # ... and those it had before, which captured graphs may still use
_workspace_lock = threading.Lock()


def _zeroed(dev, nbytes):
    """Zeroed device memory.  Inside a capture torch's allocator would give the graph's, and
    the zeroing would be left to the replays: there it is made beside the capture, at once."""
    if torch.cuda.is_current_stream_capturing():
        return _load_marshal().zeroed(nbytes, dev.index)
    return torch.zeros(nbytes, dtype=torch.uint8, device=dev)


def workspace(device=None, nbytes: int = 256) -> torch.Tensor:
    """The per-device workspace (zeroed when made), at least ``nbytes`` long.  Where a
    longer one replaces it, it stays allocated, for the graphs captured with it
    (gge_read_device_status reads both); each is twice as long as the last, so those kept
    take no more than the one in use."""
    dev = _cuda_device(device)
    ws = _workspaces.get(dev.index)
    if ws is not None and ws.numel() >= nbytes:
        return ws
    with _workspace_lock:
        ws = _workspaces.get(dev.index)
        if ws is None or ws.numel() < nbytes:
            new = _zeroed(dev, max(nbytes, 256, 2 * ws.numel() if ws is not None else 0))
            if ws is not None:
                _replaced.setdefault(dev.index, []).append(ws)
            _workspaces[dev.index] = ws = new
        return ws


def new_workspace(device=None, nbytes: int = 32 << 20) -> torch.Tensor:
    """A zeroed workspace of its own, for calls that may run at the same time on
    different streams: each such stream passes its own (``workspace=``) to the
    entry points, since by default every call on a device shares the one that
    ``workspace()`` keeps (its status words, scheduler counters and split tickets)."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=dev)


_shared_workspace = workspace


def _ws(device, need, given):
    """The caller's workspace (checked), or the shared per-device one."""
    if given is None:
        return _shared_workspace(device, need)
    if given.dtype != torch.uint8 or given.device != device or not given.is_contiguous():
        raise ValueError("workspace: a contiguous uint8 tensor on the outputs' device")
    return given


# gge_config.flags bits (include/gge.h)
FLAGS = {
    "tile_counts": 1,          # count tile visits into tile_counts
    "test_drop_acc_full": 2,   # test hook: the epilogue's accumulator wait runs out
    "dynamic_sched": 4,        # tiles claimed from a counter in the workspace
    "direct_stores": 8,        # epilogue stores without shared-memory staging
    "no_split": 32,            # never split the last wave along K
    "raster_n": 128,           # raster bands of n-tiles
    "clc_sched": 256,          # cluster launch control: steal the tiles of unlaunched clusters
    "swap_ab": 512,            # compute D^T = B A^T (outputs stored transposed by the kernel)
    "k_serpentine": 1024,      # odd waves walk K backwards (L2 reuse across waves)
}
RESERVED_FLAGS = 16 | 64       # a call that sets one of these is rejected


def make_config(tile_n=0, num_ctas=0, raster_band=0, stages=0, flags=0, tile_counts=None,
                timeout_ns=0, cta_group=0, batch_idx_permute=None):
    """batch_idx_permute: None or a device int32 tensor [L] (a permutation of 0..L-1)."""
    return GgeConfig(tile_n, num_ctas, raster_band, stages, flags, cta_group,
                     ctypes.c_void_p(tile_counts.data_ptr()) if tile_counts is not None else None,
                     timeout_ns,
                     ctypes.c_void_p(batch_idx_permute.data_ptr())
                     if batch_idx_permute is not None else None)


def make_args(A, B, C=None, D=None, PostAct=None, alpha=1.0, beta=1.0, act="none",
              alpha_dev=None, beta_dev=None, config=None, a_kind="mk"):
    keep = []

    def opt(t):
        if t is None:
            return None
        v = view(t, "mn")
        keep.append(v)
        return ctypes.pointer(v)

    args = GgeGemmArgs()
    args.A = view(A, a_kind)
    args.B = view(B, "nk")
    args.C, args.D, args.PostAct = opt(C), opt(D), opt(PostAct)
    args.alpha, args.beta = float(alpha), float(beta)
    args.alpha_dev = ctypes.c_void_p(alpha_dev.data_ptr()) if alpha_dev is not None else None
    args.beta_dev = ctypes.c_void_p(beta_dev.data_ptr()) if beta_dev is not None else None
    args.act = ACT[act]
    args.config = ctypes.pointer(config) if config is not None else None
    args._keep = (keep, config)
    return args


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _check(code, where):
    if code != 0:
        raise GgeError(code, where)


def _current(dev):
    """The library plans and launches on the current device: makes ``dev`` that one (a host
    tensor's makes no difference) for the length of a with statement."""
    if dev.type != "cuda" or dev.index is None or torch.cuda.current_device() == dev.index:
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def _on_device_of(name):
    """Calls the function with the device of its argument ``name``, a tensor, current."""
    def wrap(f):
        at = list(inspect.signature(f).parameters).index(name)

        @functools.wraps(f)
        def call(*args, **kw):
            dev = getattr(args[at] if len(args) > at else kw.get(name), "device", None)
            if dev is None or dev.type != "cuda" or torch.cuda.current_device() == dev.index:
                return f(*args, **kw)
            with torch.cuda.device(dev):
                return f(*args, **kw)
        return call
    return wrap


# ------------------------------------------------------------- entry points

@_on_device_of("A")
def gge_gemm(A, B, D, C=None, alpha=1.0, beta=1.0, alpha_dev=None, beta_dev=None, config=None,
             workspace=None):
    """D = alpha * A @ B^T + beta * C.  A (L,M,K)/(M,K), B (L,N,K)/(N,K), D (L,M,N)/(M,N).
    workspace: optional buffer of the caller's (see new_workspace)."""
    lib = load()
    args = make_args(A, B, C=C, D=D, alpha=alpha, beta=beta, alpha_dev=alpha_dev,
                     beta_dev=beta_dev, config=config)
    ws = _ws(D.device, lib.gge_workspace_size(ctypes.byref(args), 0), workspace)
    _check(lib.gge_gemm(ctypes.byref(args), ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                        _stream(D)), "gge_gemm")


@_on_device_of("A")
def gge_gemm_act(A, B, PostAct, act, D=None, C=None, alpha=1.0, beta=1.0, alpha_dev=None,
                 beta_dev=None, config=None, workspace=None):
    """D (optional) and PostAct = act(alpha * A @ B^T + beta * C)."""
    lib = load()
    args = make_args(A, B, C=C, D=D, PostAct=PostAct, alpha=alpha, beta=beta, act=act,
                     alpha_dev=alpha_dev, beta_dev=beta_dev, config=config)
    ws = _ws(PostAct.device, lib.gge_workspace_size(ctypes.byref(args), 0), workspace)
    _check(lib.gge_gemm_act(ctypes.byref(args), ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                            _stream(PostAct)), "gge_gemm_act")


@_on_device_of("A")
def gge_gemm_dact(A, B, PreAct, D, act, PostAct=None, config=None, workspace=None):
    """Backward activation epilogue: D = act'(PreAct) * (A @ B^T), PostAct = act(PreAct)."""
    lib = load()
    args = make_args(A, B, C=PreAct, D=D, PostAct=PostAct, act=act, config=config)
    ws = _ws(D.device, lib.gge_workspace_size(ctypes.byref(args), 0), workspace)
    _check(lib.gge_gemm_dact(ctypes.byref(args), ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                             _stream(D)), "gge_gemm_dact")


@_on_device_of("A")
def gge_gemm_act_static_scratch(A, B, PostAct, act, D=None, C=None, alpha=1.0, beta=1.0,
                                config=None):
    """gge_gemm_act for callers that cannot allocate: no workspace argument, the
    library's own fixed scratch area is used (see include/gge.h)."""
    lib = load()
    args = make_args(A, B, C=C, D=D, PostAct=PostAct, alpha=alpha, beta=beta, act=act,
                     config=config)
    _check(lib.gge_gemm_act_static_scratch(ctypes.byref(args), _stream(PostAct)),
           "gge_gemm_act_static_scratch")


@_on_device_of("A")
def gge_gemm_varlen_m(A, B, cu_seqlens_m, D=None, PostAct=None, act="none", C=None, alpha=1.0,
                      beta=1.0, config=None, workspace=None):
    """Varlen-M grouped GEMM: A (total_M, K), B (G, N, K), cu_seqlens_m int32 (G+1,) on device."""
    lib = load()
    out = D if D is not None else PostAct
    args = make_args(A, B, C=C, D=D, PostAct=PostAct, alpha=alpha, beta=beta, act=act,
                     config=config)
    ws = _ws(out.device, 256, workspace)
    G = cu_seqlens_m.numel() - 1
    _check(lib.gge_gemm_varlen_m(ctypes.byref(args), ctypes.c_void_p(cu_seqlens_m.data_ptr()), G,
                                 ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream(out)),
           "gge_gemm_varlen_m")


@_on_device_of("A")
def gge_gemm_varlen_k(A, B, cu_seqlens_k, D=None, PostAct=None, act="none", C=None, alpha=1.0,
                      beta=1.0, config=None, workspace=None):
    """Varlen-K grouped GEMM: A (M, total_K), B (N, total_K), cu_seqlens_k int32 (G+1,) on
    device; C / D / PostAct (G, M, N).  Group g contracts K columns cu[g] .. cu[g+1]-1."""
    lib = load()
    out = D if D is not None else PostAct
    args = make_args(A, B, C=C, D=D, PostAct=PostAct, alpha=alpha, beta=beta, act=act,
                     config=config)
    G = cu_seqlens_k.numel() - 1
    need = lib.gge_workspace_size_varlen_k(ctypes.byref(args), G)
    ws = _ws(out.device, need, workspace)
    _check(lib.gge_gemm_varlen_k(ctypes.byref(args), ctypes.c_void_p(cu_seqlens_k.data_ptr()), G,
                                 ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream(out)),
           "gge_gemm_varlen_k")


@_on_device_of("A_src")
def gge_gemm_gather_k(A_src, B, a_idx, cu_seqlens_k, D=None, PostAct=None, act="none", C=None,
                      alpha=1.0, beta=1.0, config=None, workspace=None):
    """Gather-K: varlen-K GEMM whose A column k is A_src[:, a_idx[k]].  A_src (M, K_src)
    M-major (e.g. X.t() of a row-major X [K_src, M]), B (N, total_K), a_idx int32
    (total_K,), cu_seqlens_k int32 (G+1,); C / D / PostAct (G, M, N)."""
    lib = load()
    out = D if D is not None else PostAct
    args = make_args(A_src, B, C=C, D=D, PostAct=PostAct, alpha=alpha, beta=beta, act=act,
                     config=config)
    G = cu_seqlens_k.numel() - 1
    ws = _ws(out.device, lib.gge_workspace_size_varlen_k(ctypes.byref(args), G), workspace)
    _check(lib.gge_gemm_gather_k(ctypes.byref(args), ctypes.c_void_p(a_idx.data_ptr()),
                                 ctypes.c_void_p(cu_seqlens_k.data_ptr()), G,
                                 ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream(out)),
           "gge_gemm_gather_k")


@_on_device_of("A_src")
def gge_gemm_gather_a(A_src, B, a_idx, cu_seqlens_m=None, D=None, PostAct=None, act="none",
                      C=None, alpha=1.0, beta=1.0, config=None, workspace=None):
    """Gather-A GEMM: effective A row r = A_src[a_idx[r]]; varlen-M when cu_seqlens_m is given."""
    lib = load()
    out = D if D is not None else PostAct
    args = make_args(A_src, B, C=C, D=D, PostAct=PostAct, alpha=alpha, beta=beta, act=act,
                     config=config)
    ws = _ws(out.device, 256, workspace)
    G = cu_seqlens_m.numel() - 1 if cu_seqlens_m is not None else 0
    cu = ctypes.c_void_p(cu_seqlens_m.data_ptr()) if cu_seqlens_m is not None else None
    _check(lib.gge_gemm_gather_a(ctypes.byref(args), ctypes.c_void_p(a_idx.data_ptr()), cu, G,
                                 ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream(out)),
           "gge_gemm_gather_a")


def _cuda_device(device):
    dev = torch.device("cuda" if device is None else device)
    return dev if dev.index is not None else torch.device("cuda", torch.cuda.current_device())


def gge_read_static_scratch_status(device=None):
    """Synchronise the current stream and return (status_name, where, tile) that
    gge_gemm_act_static_scratch calls recorded in the library's area; clears it."""
    dev = _cuda_device(device)
    with _current(dev):
        lib = load()
        detail = (c_i32 * 2)()
        stream = ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)
        code = lib.gge_read_static_scratch_status(stream, detail)
    return STATUS.get(code, str(code)), detail[0], detail[1]


def gge_read_device_status(device=None, workspace=None):
    """Synchronise the current stream and return (status_name, where, tile) recorded in
    the shared per-device workspace or one that it replaced (or in ``workspace``, a
    caller's); clears it."""
    dev = _cuda_device(device) if workspace is None else workspace.device
    with _current(dev):
        lib = load()
        places = [workspace] if workspace is not None else [_shared_workspace(dev)] + _replaced.get(dev.index, [])
        detail = (c_i32 * 2)()
        for ws in places:
            code = lib.gge_read_device_status(ctypes.c_void_p(ws.data_ptr()), _stream(ws), detail)
            if code != 0:
                break
    return STATUS.get(code, str(code)), detail[0], detail[1]


FORM = {"default": 0, "gather_a": 1, "varlen_k": 2, "gather_k": 3}


@_on_device_of("A")
def gge_plan(A, B, C=None, D=None, PostAct=None, act="none", num_groups=0, gather=False,
             config=None, form=None):
    """The launch plan; form: 'default' (plain / varlen-M), 'gather_a' or 'varlen_k'."""
    lib = load()
    args = make_args(A, B, C=C, D=D, PostAct=PostAct, act=act, config=config)
    info = GgePlanInfo()
    f = FORM[form] if form is not None else (1 if gather else 0)
    code = lib.gge_plan(ctypes.byref(args), num_groups, f, ctypes.byref(info))
    _check(code, "gge_plan")
    return {k: getattr(info, k) for k, _ in GgePlanInfo._fields_}


# ------------------------------------------------------------------ autotuning

OP = {"gemm": 0, "dact": 1, "varlen_m": 2, "gather_a": 3, "varlen_k": 4, "gather_k": 5}
_CFG_KEYS = ("tile_n", "num_ctas", "raster_band", "stages", "flags", "cta_group")


def config_dict(c: GgeConfig) -> dict:
    return {k: getattr(c, k) for k in _CFG_KEYS}


def _tune_args(op, A, B, C, D, PostAct, act, alpha, beta, config):
    if op == "dact":   # the backward epilogue reads the pre-activation from C
        return make_args(A, B, C=C, D=D, PostAct=PostAct, act=act, config=config)
    return make_args(A, B, C=C, D=D, PostAct=PostAct, alpha=alpha, beta=beta, act=act,
                     config=config)


@_on_device_of("A")
def gge_tune_candidates(op, A, B, C=None, D=None, PostAct=None, act="none", num_groups=0,
                        config=None):
    """The launch configurations gge_autotune would time for this problem (host only)."""
    lib = load()
    args = _tune_args(op, A, B, C, D, PostAct, act, 1.0, 1.0, config)
    out = (GgeConfig * 64)()
    n = lib.gge_tune_candidates(ctypes.byref(args), OP[op], num_groups, out, 64)
    return [config_dict(out[i]) for i in range(min(n, 64))]


@_on_device_of("A")
def gge_autotune(op, A, B, idx=None, cu=None, C=None, D=None, PostAct=None, act="none",
                 alpha=1.0, beta=1.0, reps=10, config=None):
    """Time every candidate launch shape of `op` on the current stream and return
    (best config as a dict, its mean time in ms).  The outputs hold the result."""
    lib = load()
    out = D if D is not None else PostAct
    args = _tune_args(op, A, B, C, D, PostAct, act, alpha, beta, config)
    G = cu.numel() - 1 if cu is not None else 0
    if op in ("varlen_k", "gather_k"):
        need = lib.gge_workspace_size_varlen_k(ctypes.byref(args), G)
    else:
        need = lib.gge_workspace_size(ctypes.byref(args), G)
    ws = workspace(out.device, need)
    best = GgeConfig()
    ms = ctypes.c_float()
    code = lib.gge_autotune(ctypes.byref(args), OP[op],
                            ctypes.c_void_p(idx.data_ptr()) if idx is not None else None,
                            ctypes.c_void_p(cu.data_ptr()) if cu is not None else None, G,
                            ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream(out), reps,
                            ctypes.byref(best), ctypes.byref(ms))
    _check(code, "gge_autotune")
    return config_dict(best), ms.value


@_on_device_of("A")
def gge_tuned_config(op, A, B, C=None, D=None, PostAct=None, act="none", num_groups=0,
                     config=None):
    """The configuration gge_autotune stored for a problem of this key, or None."""
    lib = load()
    args = _tune_args(op, A, B, C, D, PostAct, act, 1.0, 1.0, config)
    c = GgeConfig()
    if lib.gge_tuned_config(ctypes.byref(args), OP[op], num_groups, ctypes.byref(c)) != 0:
        return None
    return config_dict(c)


# ------------------------------------------------- low-precision linear layers

MX_FORMAT = {"mxfp8": 0, "mxfp4": 1, "nvfp4": 2}
_MX_BLOCK = (32, 32, 16)


def _mx_row_bytes(fmt, cols):
    return (cols + 31) // 32 * (32 if fmt == 0 else 16)


def _mx_kgroups(fmt, cols):
    block = _MX_BLOCK[fmt]
    return ((cols + block - 1) // block + 3) // 4


def _mx_scale_bytes(fmt, rows, cols):
    return (rows + 127) // 128 * _mx_kgroups(fmt, cols) * 512


class MxTensor:
    """A microscaled matrix (gge_mx_tensor): codes (rows, bytes) or (batch, rows, bytes)
    uint8, scales a contiguous uint8 tensor of gge_mx_scale_bytes a batch, tensor_scale None
    or a one-element fp32 tensor (nvfp4), all on one CUDA device.  ``c`` holds the C struct
    as bytes, made once: its tensors' contents may change, the tensors may not (another tensor
    scale is another MxTensor over the same codes and scales)."""

    __slots__ = ("_format", "_tensor_scale", "_device", "_c", "_codes", "_scales", "_buffer",
                 "_batched")

    def __init__(self, codes, scales, format, rows, cols, tensor_scale=None):
        self._c = (_marshal or _load_marshal()).mx_wrap(codes, scales, MX_FORMAT[format], rows, cols,
                                                        tensor_scale)
        self._device = codes.device
        self._format, self._tensor_scale = format, tensor_scale
        self._codes, self._scales = codes, scales

    c = property(operator.attrgetter("_c"))
    device = property(operator.attrgetter("_device"))
    format = property(operator.attrgetter("_format"))
    tensor_scale = property(operator.attrgetter("_tensor_scale"))

    def _struct(self):
        return GgeMxTensor.from_buffer_copy(self._c)

    @property
    def rows(self):
        return self._struct().rows

    @property
    def cols(self):
        return self._struct().cols

    @property
    def batch(self):
        return self._struct().batch

    @property
    def codes(self):
        if self._codes is None:   # mx_empty: a view of its one buffer, made when asked for
            c = self._struct()
            row = c.stride_row
            if self._batched:
                self._codes = self._buffer.as_strided((c.batch, c.rows, row), (c.stride_batch, row, 1))
            else:
                self._codes = self._buffer.as_strided((c.rows, row), (row, 1))
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            c = self._struct()
            self._scales = self._buffer.as_strided((c.batch * c.scale_stride_batch,), (1,),
                                                   (c.scales or 0) - (c.codes or 0))
        return self._scales


def mx_empty(rows, cols, format, device=None, batch=None, tensor_scale=None):
    """An MxTensor with room for (rows, cols) or (batch, rows, cols) values on a CUDA device:
    its codes and scales share one allocation."""
    fmt = MX_FORMAT[format]
    if device is None or device.__class__ is not torch.device or device.index is None:
        device = torch.device("cuda" if device is None else device)
        if device.index is None:
            device = torch.device(device.type, torch.cuda.current_device())
    if device.type != "cuda":
        raise ValueError("mx_empty: not a CUDA device")
    if rows < 0 or cols < 0 or (batch is not None and batch < 1):
        raise ValueError("mx_empty: rows and cols may not be negative, batch not below 1")
    row, per = _mx_row_bytes(fmt, cols), _mx_scale_bytes(fmt, rows, cols)
    b = 1 if batch is None else batch
    start = (b * rows * row + 511) & ~511
    q = MxTensor.__new__(MxTensor)
    q._buffer, q._c = (_marshal or _load_marshal()).mx_alloc(
        start + b * per, start, device.index, fmt, rows, cols, 0 if batch is None else batch, row, per,
        tensor_scale)
    q._device, q._format, q._tensor_scale = device, format, tensor_scale
    q._codes = q._scales = None
    q._batched = batch is not None
    return q


def _shared(device, need):
    """The shared workspace of a device, at least `need` bytes."""
    ws = _workspaces.get(device.index)
    if ws is None or ws.numel() < need:
        ws = _shared_workspace(device, need)
    return ws


def _on(Q, device):
    """The C struct of an MxTensor that has to be on a device."""
    if Q._device != device:
        raise ValueError("MxTensor: tensors on different devices")
    return Q._c


def gge_mx_quantize(X, Q, values=None):
    """Q (an MxTensor) = X quantised; X (rows, cols) or (batch, rows, cols), row-major or a
    transposed view.  values: optional output, the numbers that the codes stand for."""
    code = (_marshal or _load_marshal()).quantize(X, _on(Q, X.device), values)
    if code:
        raise GgeError(code, "gge_mx_quantize")


def gge_mx_dequantize(Q, Y):
    """Y (bf16, f16 or f32) = the numbers that Q's codes stand for."""
    code = (_marshal or _load_marshal()).dequantize(_on(Q, Y.device), Y)
    if code:
        raise GgeError(code, "gge_mx_dequantize")


def gge_gemm_mx(A, B, D=None, C=None, PostAct=None, act="none", alpha=1.0, beta=1.0,
                alpha_dev=None, beta_dev=None, config=None, workspace=None):
    """D = alpha * A @ B^T + beta * C and / or PostAct = act(same) of MxTensors A (M, K) and
    B (N, K) (or batched), their tensor scales included."""
    dev = A._device
    ws = _shared(dev, 256) if workspace is None else _ws(dev, 256, workspace)
    code = (_marshal or _load_marshal()).gemm_mx(
        A._c, _on(B, dev), dev.index, D, C, PostAct, ACT[act], alpha, beta, alpha_dev, beta_dev,
        ctypes.addressof(config) if config is not None else 0, ws, False)
    if code:
        raise GgeError(code, "gge_gemm_mx")


def gge_gemm_mx_dact(A, B, PreAct, D, act, PostAct=None, config=None, workspace=None):
    """Backward activation epilogue on MxTensors: D = act'(PreAct) * (A @ B^T), PostAct =
    act(PreAct)."""
    dev = A._device
    ws = _shared(dev, 256) if workspace is None else _ws(dev, 256, workspace)
    code = (_marshal or _load_marshal()).gemm_mx(
        A._c, _on(B, dev), dev.index, D, PreAct, PostAct, ACT[act], 1.0, 1.0, None, None,
        ctypes.addressof(config) if config is not None else 0, ws, True)
    if code:
        raise GgeError(code, "gge_gemm_mx_dact")


def gge_rmsnorm(X, weight, Y=None, residual=None, residual_out=None, Q=None, values=None,
                inv_rms=None, eps=1e-6):
    """h = X + residual (rounded to X's type, written to residual_out), inv_rms = 1 / sqrt(mean
    h^2 + eps) a row, Y = h * inv_rms * weight; Q (an MxTensor) = the same quantised, values =
    the numbers that Q's codes stand for.  X (rows, cols); every output is optional."""
    code = (_marshal or _load_marshal()).rmsnorm(
        X, weight, Y, residual, residual_out, _on(Q, X.device) if Q is not None else None, values,
        inv_rms, eps)
    if code:
        raise GgeError(code, "gge_rmsnorm")


def gge_rmsnorm_bwd(dY, H, weight, inv_rms, dX, dW=None, dH=None, workspace=None):
    """Backward of gge_rmsnorm: dX (the gradient of X and of the residual) from dY, the saved H
    (residual_out, or X) and inv_rms; dW (fp32, optional); dH the gradient reaching H directly.
    dW's partial sums take gge_workspace_size_rmsnorm_bwd(cols) bytes: memory of the call's own
    from torch's allocator on the current stream, or the caller's ``workspace``."""
    ws = None if workspace is None else _ws(dY.device, 0, workspace)
    code = (_marshal or _load_marshal()).rmsnorm_bwd(dY, H, weight, inv_rms, dX, dW, dH, ws)
    if code:
        raise GgeError(code, "gge_rmsnorm_bwd")
