// Argument marshalling of the low-precision entry points for Python: torch tensors
// in, the C structs of include/gge.h out, one call each.  The checks are those of
// the arguments' Python side (types, devices, shapes of the plain vectors); the
// library checks the rest.  A call this way costs 2 to 3 us of host time, through
// ctypes 6 to 9, which is what a small norm or product takes on the GPU.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAException.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include "../../../include/gge.h"

namespace {

int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return GGE_BF16;
    case at::kHalf: return GGE_F16;
    case at::kFloat8_e4m3fn: return GGE_E4M3;
    case at::kFloat8_e5m2: return GGE_E5M2;
    case at::kFloat: return GGE_F32;
    default: return -1;
  }
}

// The tensor of a Python object on device `dev` (-1: any CUDA device), or NULL with an
// exception set.
const at::Tensor* tensor(PyObject* o, const char* kind, int dev) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: expected a tensor", kind);
    return nullptr;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || (dev >= 0 && t.get_device() != dev)) {
    PyErr_Format(PyExc_ValueError, t.is_cuda() ? "%s: tensors on different devices" : "%s: not a CUDA tensor", kind);
    return nullptr;
  }
  return &t;
}

// A (rows, cols) or (batch, rows, cols) tensor as a C view.  0: None (allowed when
// `optional`), 1: filled, -1: an exception is set.
int view(PyObject* o, const char* kind, int dev, bool optional, gge_tensor* out, bool flat = false) {
  if (optional && o == Py_None) return 0;
  const at::Tensor* t = tensor(o, kind, dev);
  if (t == nullptr) return -1;
  const int64_t dim = t->dim();
  if (dim != 2 && (dim != 3 || flat)) {
    PyErr_Format(PyExc_ValueError, flat ? "%s: expected a 2-D tensor" : "%s: expected a 2-D or 3-D tensor", kind);
    return -1;
  }
  const int code = dtype_code(t->scalar_type());
  if (code < 0) {
    PyErr_Format(PyExc_TypeError, "%s: unsupported dtype", kind);
    return -1;
  }
  const auto size = t->sizes();
  const auto stride = t->strides();
  const int b = dim == 3 ? 1 : 0;
  *out = gge_tensor{t->data_ptr(), code, 0, size[b], size[b + 1], b ? size[0] : 1,
                    stride[b], stride[b + 1], b ? stride[0] : 0};
  return 1;
}

// A contiguous vector of n values (of `type`, if it is not Undefined).
int vector(PyObject* o, const char* kind, int dev, bool optional, int64_t n, at::ScalarType type, void** out,
           int* code = nullptr) {
  *out = nullptr;
  if (optional && o == Py_None) return 0;
  const at::Tensor* t = tensor(o, kind, dev);
  if (t == nullptr) return -1;
  const bool typed = type != at::ScalarType::Undefined;
  if (t->numel() != n || !t->is_contiguous() || (typed && t->scalar_type() != type)) {
    PyErr_Format(PyExc_ValueError, "%s: expected %lld contiguous values%s", kind, static_cast<long long>(n),
                 typed ? " of the right type" : "");
    return -1;
  }
  if (code != nullptr) {
    *code = dtype_code(t->scalar_type());
    if (*code < 0) {
      PyErr_Format(PyExc_TypeError, "%s: unsupported dtype", kind);
      return -1;
    }
  }
  *out = t->data_ptr();
  return 1;
}

// The gge_mx_tensor that an MxTensor carries as bytes.
const gge_mx_tensor* mx(PyObject* o, bool optional) {
  if (optional && o == Py_None) return nullptr;
  if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) != sizeof(gge_mx_tensor)) {
    PyErr_SetString(PyExc_TypeError, "expected an MxTensor");
    return nullptr;
  }
  return reinterpret_cast<const gge_mx_tensor*>(PyBytes_AS_STRING(o));
}

gge_stream_t stream(int dev) {
  return reinterpret_cast<gge_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
}

bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

int device_of(PyObject* o, const char* kind) {
  const at::Tensor* t = tensor(o, kind, -1);
  return t == nullptr ? -1 : static_cast<int>(t->get_device());
}

// Every call into the library goes through this one: with the tensors' device current (the
// library plans and launches on that) and on its current stream, `st`; without the GIL.
#define GGE_CALL(dev, expr)                                                              \
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));                  \
  gge_stream_t st = stream(dev);                                                         \
  gge_status code;                                                                       \
  Py_BEGIN_ALLOW_THREADS;                                                                \
  code = (expr);                                                                         \
  Py_END_ALLOW_THREADS;                                                                  \
  return PyLong_FromLong(code)

// mx_alloc(bytes, start, device, format, rows, cols, batch or 0, row bytes, scale bytes a batch,
// tensor_scale) -> (buffer, struct bytes): codes at the buffer's start, scales at `start`
PyObject* mx_alloc(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 10)) return nullptr;
  const int64_t bytes = PyLong_AsLongLong(a[0]), start = PyLong_AsLongLong(a[1]);
  const int64_t dev = PyLong_AsLongLong(a[2]);
  const int format = static_cast<int>(PyLong_AsLong(a[3]));
  const int64_t rows = PyLong_AsLongLong(a[4]), cols = PyLong_AsLongLong(a[5]), batch = PyLong_AsLongLong(a[6]);
  const int64_t row = PyLong_AsLongLong(a[7]), per = PyLong_AsLongLong(a[8]);
  if (PyErr_Occurred()) return nullptr;
  void* scale = nullptr;
  if (vector(a[9], "tensor_scale", static_cast<int>(dev), true, 1, at::kFloat, &scale) < 0) return nullptr;
  at::Tensor buf = at::empty({bytes}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)));
  uint8_t* p = static_cast<uint8_t*>(buf.data_ptr());
  const gge_mx_tensor m{p, p + start, static_cast<const float*>(scale), format, 0, rows, cols,
                        batch > 0 ? batch : 1, row, batch > 0 ? rows * row : 0, per};
  PyObject* s = PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&m), sizeof(m));
  if (s == nullptr) return nullptr;
  PyObject* t = THPVariable_Wrap(std::move(buf));
  if (t == nullptr) {
    Py_DECREF(s);
    return nullptr;
  }
  PyObject* r = PyTuple_Pack(2, t, s);
  Py_DECREF(t);
  Py_DECREF(s);
  return r;
  END_HANDLE_TH_ERRORS
}

// mx_wrap(codes, scales, format, rows, cols, tensor_scale) -> struct bytes
PyObject* mx_wrap(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 6)) return nullptr;
  const at::Tensor* codes = tensor(a[0], "codes", -1);
  if (codes == nullptr) return nullptr;
  const int dev = static_cast<int>(codes->get_device());
  const at::Tensor* scales = tensor(a[1], "scales", dev);
  if (scales == nullptr) return nullptr;
  const int format = static_cast<int>(PyLong_AsLong(a[2]));
  const int64_t rows = PyLong_AsLongLong(a[3]), cols = PyLong_AsLongLong(a[4]);
  if (PyErr_Occurred()) return nullptr;
  void* scale = nullptr;
  if (vector(a[5], "tensor_scale", dev, true, 1, at::kFloat, &scale) < 0) return nullptr;
  if (codes->scalar_type() != at::kByte || scales->scalar_type() != at::kByte) {
    PyErr_SetString(PyExc_TypeError, "MxTensor: codes and scales are uint8 tensors");
    return nullptr;
  }
  const int64_t dim = codes->dim();
  if (dim != 2 && dim != 3) {
    PyErr_SetString(PyExc_ValueError, "MxTensor: codes are 2-D or 3-D (batch first)");
    return nullptr;
  }
  const int b = dim == 3 ? 1 : 0;
  const int64_t batch = b ? codes->size(0) : 1;
  const int64_t per = static_cast<int64_t>(gge_mx_scale_bytes(format, rows, cols));
  if (codes->size(b) != rows || codes->size(b + 1) != static_cast<int64_t>(gge_mx_row_bytes(format, cols)) ||
      (codes->stride(b + 1) != 1 && codes->numel() > 0)) {
    PyErr_SetString(PyExc_ValueError, "MxTensor: codes do not match rows, cols and format");
    return nullptr;
  }
  if (scales->numel() != batch * per || !scales->is_contiguous()) {
    PyErr_SetString(PyExc_ValueError, "MxTensor: scales do not match rows, cols and format");
    return nullptr;
  }
  const gge_mx_tensor m{codes->data_ptr(), scales->data_ptr(), static_cast<const float*>(scale), format, 0,
                        rows, cols, batch, codes->stride(b), b ? codes->stride(0) : 0, per};
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&m), sizeof(m));
  END_HANDLE_TH_ERRORS
}

// quantize(X, Q, values)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 3)) return nullptr;
  const int dev = device_of(a[0], "X");
  gge_tensor x, v;
  const gge_mx_tensor* q = mx(a[1], false);
  if (dev < 0 || q == nullptr || view(a[0], "X", dev, false, &x) < 0) return nullptr;
  const int has = view(a[2], "values", dev, true, &v);
  if (has < 0) return nullptr;
  GGE_CALL(dev, gge_mx_quantize(&x, q, has ? &v : nullptr, st));
  END_HANDLE_TH_ERRORS
}

// dequantize(Q, Y)
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 2)) return nullptr;
  const int dev = device_of(a[1], "Y");
  gge_tensor y;
  const gge_mx_tensor* q = mx(a[0], false);
  if (dev < 0 || q == nullptr || view(a[1], "Y", dev, false, &y) < 0) return nullptr;
  GGE_CALL(dev, gge_mx_dequantize(q, &y, st));
  END_HANDLE_TH_ERRORS
}

// gemm_mx(A, B, device, D, C, PostAct, act, alpha, beta, alpha_dev, beta_dev, config address or 0, workspace,
// backward epilogue)
PyObject* gemm_mx(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 14)) return nullptr;
  const gge_mx_tensor* A = mx(a[0], false);
  if (A == nullptr) return nullptr;
  const gge_mx_tensor* B = mx(a[1], false);
  if (B == nullptr) return nullptr;
  const int dev = static_cast<int>(PyLong_AsLong(a[2]));
  gge_tensor d, c, p;
  const int hd = view(a[3], "D", dev, true, &d);
  if (hd < 0) return nullptr;
  const int hc = view(a[4], "C", dev, true, &c);
  if (hc < 0) return nullptr;
  const int hp = view(a[5], "PostAct", dev, true, &p);
  if (hp < 0) return nullptr;
  gge_gemm_mx_args g;
  g.A = *A;
  g.B = *B;
  g.D = hd ? &d : nullptr;
  g.C = hc ? &c : nullptr;
  g.PostAct = hp ? &p : nullptr;
  g.act = static_cast<int32_t>(PyLong_AsLong(a[6]));
  g.alpha = static_cast<float>(PyFloat_AsDouble(a[7]));
  g.beta = static_cast<float>(PyFloat_AsDouble(a[8]));
  g.reserved = 0;
  void *alpha = nullptr, *beta = nullptr;
  if (vector(a[9], "alpha_dev", dev, true, 1, at::kFloat, &alpha) < 0 ||
      vector(a[10], "beta_dev", dev, true, 1, at::kFloat, &beta) < 0)
    return nullptr;
  g.alpha_dev = static_cast<const float*>(alpha);
  g.beta_dev = static_cast<const float*>(beta);
  g.config = static_cast<const gge_config*>(PyLong_AsVoidPtr(a[11]));
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor* ws = tensor(a[12], "workspace", dev);
  if (ws == nullptr) return nullptr;
  void* wp = ws->data_ptr();
  const size_t wn = static_cast<size_t>(ws->numel());
  const bool dact = PyObject_IsTrue(a[13]) == 1;
  GGE_CALL(dev, dact ? gge_gemm_mx_dact(&g, wp, wn, st) : gge_gemm_mx(&g, wp, wn, st));
  END_HANDLE_TH_ERRORS
}

// rmsnorm(X, weight, Y, residual, residual_out, Q or None, values, inv_rms, eps)
PyObject* rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 9)) return nullptr;
  const int dev = device_of(a[0], "X");
  gge_rmsnorm_args g;
  if (dev < 0 || view(a[0], "X", dev, false, &g.x, true) < 0) return nullptr;
  void *w = nullptr, *inv = nullptr;
  int wt = 0;
  if (vector(a[1], "weight", dev, false, g.x.cols, at::ScalarType::Undefined, &w, &wt) < 0) return nullptr;
  gge_tensor y, r, h, v;
  const int hy = view(a[2], "Y", dev, true, &y);
  if (hy < 0) return nullptr;
  const int hr = view(a[3], "residual", dev, true, &r);
  if (hr < 0) return nullptr;
  const int hh = view(a[4], "residual_out", dev, true, &h);
  if (hh < 0) return nullptr;
  const gge_mx_tensor* q = mx(a[5], true);
  if (q == nullptr && a[5] != Py_None) return nullptr;
  const int hv = view(a[6], "values", dev, true, &v);
  if (hv < 0) return nullptr;
  if (vector(a[7], "inv_rms", dev, true, g.x.rows, at::kFloat, &inv) < 0) return nullptr;
  g.eps = static_cast<float>(PyFloat_AsDouble(a[8]));
  if (PyErr_Occurred()) return nullptr;
  g.residual = hr ? &r : nullptr;
  g.residual_out = hh ? &h : nullptr;
  g.y = hy ? &y : nullptr;
  g.q = q;
  g.values = hv ? &v : nullptr;
  g.weight = w;
  g.weight_dtype = wt;
  g.inv_rms = static_cast<float*>(inv);
  GGE_CALL(dev, gge_rmsnorm(&g, st));
  END_HANDLE_TH_ERRORS
}

// rmsnorm_bwd(dY, H, weight, inv_rms, dX, dW, dH, workspace or None)
PyObject* rmsnorm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 8)) return nullptr;
  const int dev = device_of(a[0], "dY");
  gge_rmsnorm_bwd_args g;
  gge_tensor dh;
  if (dev < 0 || view(a[0], "dY", dev, false, &g.dy, true) < 0 || view(a[1], "H", dev, false, &g.h, true) < 0 ||
      view(a[4], "dX", dev, false, &g.dx, true) < 0)
    return nullptr;
  void *w = nullptr, *inv = nullptr, *dw = nullptr;
  int wt = 0;
  if (vector(a[2], "weight", dev, false, g.dy.cols, at::ScalarType::Undefined, &w, &wt) < 0 ||
      vector(a[3], "inv_rms", dev, false, g.dy.rows, at::kFloat, &inv) < 0 ||
      vector(a[5], "dW", dev, true, g.dy.cols, at::kFloat, &dw) < 0)
    return nullptr;
  const int hh = view(a[6], "dH", dev, true, &dh);
  if (hh < 0) return nullptr;
  g.dh = hh ? &dh : nullptr;
  g.weight = w;
  g.weight_dtype = wt;
  g.reserved = 0;
  g.inv_rms = static_cast<const float*>(inv);
  g.dweight = static_cast<float*>(dw);
  // the partial sums' memory: the caller's, or this call's own.  That is handed back at the
  // end, for the stream's later kernels, and inside a capture belongs to the graph
  void* wp = nullptr;
  size_t wn = 0;
  at::Tensor own;
  if (a[7] != Py_None) {
    const at::Tensor* ws = tensor(a[7], "workspace", dev);
    if (ws == nullptr) return nullptr;
    wp = ws->data_ptr();
    wn = static_cast<size_t>(ws->numel());
  } else if (dw != nullptr) {
    const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(dev));
    wn = gge_workspace_size_rmsnorm_bwd(g.dy.cols);
    own = at::empty({static_cast<int64_t>(wn)},
                    at::TensorOptions().dtype(at::kByte).device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)));
    wp = own.data_ptr();
  }
  GGE_CALL(dev, gge_rmsnorm_bwd(&g, wp, wn, st));
  END_HANDLE_TH_ERRORS
}

// zeroed(bytes, device) -> uint8 tensor that is zeroed when this returns and never given
// back, also while a stream is captured (the calls are no part of the capture).
PyObject* zeroed(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 2)) return nullptr;
  const int64_t bytes = PyLong_AsLongLong(a[0]), dev = PyLong_AsLongLong(a[1]);
  if (PyErr_Occurred()) return nullptr;
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  const c10::cuda::CUDAStreamCaptureModeGuard relaxed(cudaStreamCaptureModeRelaxed);
  void* p = nullptr;
  C10_CUDA_CHECK(cudaMalloc(&p, static_cast<size_t>(bytes)));
  cudaStream_t st = nullptr;
  C10_CUDA_CHECK(cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking));
  const cudaError_t set = cudaMemsetAsync(p, 0, static_cast<size_t>(bytes), st);
  const cudaError_t done = cudaStreamSynchronize(st);
  C10_CUDA_CHECK(cudaStreamDestroy(st));
  C10_CUDA_CHECK(set);
  C10_CUDA_CHECK(done);
  return THPVariable_Wrap(at::from_blob(
      p, {bytes}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, static_cast<c10::DeviceIndex>(dev))));
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef kMethods[] = {method<mx_alloc>("mx_alloc"), method<mx_wrap>("mx_wrap"), method<quantize>("quantize"),
                          method<dequantize>("dequantize"), method<gemm_mx>("gemm_mx"),
                          method<rmsnorm>("rmsnorm"), method<rmsnorm_bwd>("rmsnorm_bwd"),
                          method<zeroed>("zeroed"),
                          {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "gge_marshal", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit_gge_marshal() {
  return PyModule_Create(&kModule);
}
