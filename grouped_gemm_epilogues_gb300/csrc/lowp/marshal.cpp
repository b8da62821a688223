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

// A workspace's size, with the tensors' device current.
size_t size_on(int64_t dev, size_t (*size_of)(int64_t), int64_t cols) {
  const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(dev));
  return size_of(cols);
}

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

// ---- 8 bits with a scale for each block of 128

// The gge_b128_tensor that a B128Tensor carries as bytes.
const gge_b128_tensor* b128(PyObject* o, bool optional) {
  if (optional && o == Py_None) return nullptr;
  if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) != sizeof(gge_b128_tensor)) {
    PyErr_SetString(PyExc_TypeError, "expected a B128Tensor");
    return nullptr;
  }
  return reinterpret_cast<const gge_b128_tensor*>(PyBytes_AS_STRING(o));
}

// A matrix in either form: a tensor or a B128Tensor's bytes.  0: None, 1: a tensor (in `t`),
// 2: codes (in `q`), -1: an exception is set.
int either(PyObject* o, const char* kind, int dev, gge_tensor* t, const gge_b128_tensor** q, bool flat = false) {
  *q = nullptr;
  if (PyBytes_Check(o)) {
    *q = b128(o, false);
    return *q == nullptr ? -1 : 2;
  }
  return view(o, kind, dev, true, t, flat);
}

// b128_wrap(codes, scales, block_rows) -> struct bytes
PyObject* b128_wrap(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 3)) return nullptr;
  const at::Tensor* codes = tensor(a[0], "codes", -1);
  if (codes == nullptr) return nullptr;
  const at::Tensor* scales = tensor(a[1], "scales", static_cast<int>(codes->get_device()));
  if (scales == nullptr) return nullptr;
  const int64_t block = PyLong_AsLongLong(a[2]);
  if (PyErr_Occurred()) return nullptr;
  const int type = dtype_code(codes->scalar_type());
  if ((type != GGE_E4M3 && type != GGE_E5M2) || scales->scalar_type() != at::kFloat) {
    PyErr_SetString(PyExc_TypeError, "B128Tensor: codes are float8_e4m3fn or float8_e5m2, scales float32");
    return nullptr;
  }
  const int64_t dim = codes->dim();
  if ((dim != 2 && dim != 3) || scales->dim() != dim) {
    PyErr_SetString(PyExc_ValueError, "B128Tensor: codes and scales are 2-D or 3-D (batch first)");
    return nullptr;
  }
  if (block != 1 && block != 128) {
    PyErr_SetString(PyExc_ValueError, "B128Tensor: block_rows is 1 or 128");
    return nullptr;
  }
  const int b = dim == 3 ? 1 : 0;
  const auto size = codes->sizes(), stride = codes->strides();
  const auto ssize = scales->sizes(), sstride = scales->strides();
  if (ssize[b] != (size[b] + block - 1) / block || ssize[b + 1] != (size[b + 1] + 127) / 128 ||
      (b && ssize[0] != size[0])) {
    PyErr_SetString(PyExc_ValueError, "B128Tensor: scales do not match the codes' blocks");
    return nullptr;
  }
  if (size[b + 1] > 1 && stride[b + 1] != 1 && codes->numel() > 0) {
    PyErr_SetString(PyExc_ValueError, "B128Tensor: a row's codes are contiguous");
    return nullptr;
  }
  const gge_b128_tensor m{codes->data_ptr(), static_cast<float*>(scales->data_ptr()), type, static_cast<int32_t>(block),
                          size[b], size[b + 1], b ? size[0] : 1, stride[b], b ? stride[0] : 0,
                          sstride[b], sstride[b + 1], b ? sstride[0] : 0};
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&m), sizeof(m));
  END_HANDLE_TH_ERRORS
}

// b128_quantize(X, Q, values)
PyObject* b128_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 3)) return nullptr;
  const int dev = device_of(a[0], "X");
  gge_tensor x, v;
  const gge_b128_tensor* q = b128(a[1], false);
  if (dev < 0 || q == nullptr || view(a[0], "X", dev, false, &x) < 0) return nullptr;
  const int has = view(a[2], "values", dev, true, &v);
  if (has < 0) return nullptr;
  GGE_CALL(dev, gge_b128_quantize(&x, q, has ? &v : nullptr, st));
  END_HANDLE_TH_ERRORS
}

// b128_transpose(X, Q, values, device)
PyObject* b128_transpose(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 4)) return nullptr;
  const gge_b128_tensor* x = b128(a[0], false);
  const gge_b128_tensor* q = x == nullptr ? nullptr : b128(a[1], false);
  const int dev = static_cast<int>(PyLong_AsLong(a[3]));
  if (q == nullptr || PyErr_Occurred()) return nullptr;
  gge_tensor v;
  const int has = view(a[2], "values", dev, true, &v);
  if (has < 0) return nullptr;
  GGE_CALL(dev, gge_b128_transpose(x, q, has ? &v : nullptr, st));
  END_HANDLE_TH_ERRORS
}

// b128_dequantize(Q, Y)
PyObject* b128_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 2)) return nullptr;
  const int dev = device_of(a[1], "Y");
  gge_tensor y;
  const gge_b128_tensor* q = b128(a[0], false);
  if (dev < 0 || q == nullptr || view(a[1], "Y", dev, false, &y) < 0) return nullptr;
  GGE_CALL(dev, gge_b128_dequantize(q, &y, st));
  END_HANDLE_TH_ERRORS
}

// gemm_b128(A, B, device, D, C, PostAct, act, alpha, beta, alpha_dev, beta_dev, config address or 0, workspace,
// backward epilogue, cu_seqlens_m or None)
PyObject* gemm_b128(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 15)) return nullptr;
  const gge_b128_tensor* A = b128(a[0], false);
  if (A == nullptr) return nullptr;
  const gge_b128_tensor* B = b128(a[1], false);
  if (B == nullptr) return nullptr;
  const int dev = static_cast<int>(PyLong_AsLong(a[2]));
  gge_tensor d, c, p;
  gge_gemm_b128_args g{};
  const int hd = either(a[3], "D", dev, &d, &g.D8);
  if (hd < 0) return nullptr;
  const int hc = either(a[4], "C", dev, &c, &g.C8);
  if (hc < 0) return nullptr;
  const int hp = either(a[5], "PostAct", dev, &p, &g.PostAct8);
  if (hp < 0) return nullptr;
  g.A = *A;
  g.B = *B;
  g.D = hd == 1 ? &d : nullptr;
  g.C = hc == 1 ? &c : nullptr;
  g.PostAct = hp == 1 ? &p : nullptr;
  g.act = static_cast<int32_t>(PyLong_AsLong(a[6]));
  g.alpha = static_cast<float>(PyFloat_AsDouble(a[7]));
  g.beta = static_cast<float>(PyFloat_AsDouble(a[8]));
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
  if (a[14] != Py_None) {
    const at::Tensor* cu = tensor(a[14], "cu_seqlens_m", dev);
    if (cu == nullptr) return nullptr;
    if (cu->scalar_type() != at::kInt || cu->dim() != 1 || cu->numel() < 2 || !cu->is_contiguous()) {
      PyErr_SetString(PyExc_ValueError, "cu_seqlens_m: expected a contiguous int32 vector of at least 2 offsets");
      return nullptr;
    }
    g.cu_seqlens_m = static_cast<const int32_t*>(cu->data_ptr());
    g.num_groups = static_cast<int32_t>(cu->numel() - 1);
  }
  GGE_CALL(dev, dact ? gge_gemm_b128_dact(&g, wp, wn, st) : gge_gemm_b128(&g, wp, wn, st));
  END_HANDLE_TH_ERRORS
}

// layernorm(X, weight, bias, Y, residual, residual_out, Q, values, H8, mean, rstd, eps)
PyObject* layernorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 12)) return nullptr;
  const int dev = device_of(a[0], "X");
  gge_layernorm_args g{};
  if (dev < 0 || view(a[0], "X", dev, false, &g.x, true) < 0) return nullptr;
  void *w = nullptr, *b = nullptr, *mean = nullptr, *rstd = nullptr;
  int wt = GGE_F32, bt = GGE_F32;
  const int hw = vector(a[1], "weight", dev, true, g.x.cols, at::ScalarType::Undefined, &w, &wt);
  if (hw < 0) return nullptr;
  const int hb = vector(a[2], "bias", dev, true, g.x.cols, at::ScalarType::Undefined, &b, &bt);
  if (hb < 0) return nullptr;
  if (hw && hb && wt != bt) {
    PyErr_SetString(PyExc_TypeError, "weight and bias are of one type");
    return nullptr;
  }
  gge_tensor y, r, h, v;
  const int hy = view(a[3], "Y", dev, true, &y);
  if (hy < 0) return nullptr;
  const int hr = view(a[4], "residual", dev, true, &r);
  if (hr < 0) return nullptr;
  const int hh = view(a[5], "residual_out", dev, true, &h);
  if (hh < 0) return nullptr;
  g.q = b128(a[6], true);
  if (g.q == nullptr && a[6] != Py_None) return nullptr;
  const int hv = view(a[7], "values", dev, true, &v);
  if (hv < 0) return nullptr;
  g.h8 = b128(a[8], true);
  if (g.h8 == nullptr && a[8] != Py_None) return nullptr;
  if (vector(a[9], "mean", dev, true, g.x.rows, at::kFloat, &mean) < 0 ||
      vector(a[10], "rstd", dev, true, g.x.rows, at::kFloat, &rstd) < 0)
    return nullptr;
  g.eps = static_cast<float>(PyFloat_AsDouble(a[11]));
  if (PyErr_Occurred()) return nullptr;
  g.residual = hr ? &r : nullptr;
  g.residual_out = hh ? &h : nullptr;
  g.y = hy ? &y : nullptr;
  g.values = hv ? &v : nullptr;
  g.weight = w;
  g.bias = b;
  g.param_dtype = hw ? wt : bt;
  g.mean = static_cast<float*>(mean);
  g.rstd = static_cast<float*>(rstd);
  GGE_CALL(dev, gge_layernorm(&g, st));
  END_HANDLE_TH_ERRORS
}

// layernorm_bwd(dY, H, weight, mean, rstd, dX, dW, dB, dH, workspace or None)
PyObject* layernorm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 10)) return nullptr;
  const int dev = device_of(a[0], "dY");
  gge_layernorm_bwd_args g{};
  gge_tensor h, dh;
  if (dev < 0 || view(a[0], "dY", dev, false, &g.dy, true) < 0 || view(a[5], "dX", dev, false, &g.dx, true) < 0)
    return nullptr;
  const int hs = either(a[1], "H", dev, &h, &g.h8, true);
  if (hs < 0) return nullptr;
  g.h = hs == 1 ? &h : nullptr;
  void *w = nullptr, *mean = nullptr, *rstd = nullptr, *dw = nullptr, *db = nullptr;
  int wt = GGE_F32;
  if (vector(a[2], "weight", dev, true, g.dy.cols, at::ScalarType::Undefined, &w, &wt) < 0 ||
      vector(a[3], "mean", dev, false, g.dy.rows, at::kFloat, &mean) < 0 ||
      vector(a[4], "rstd", dev, false, g.dy.rows, at::kFloat, &rstd) < 0 ||
      vector(a[6], "dW", dev, true, g.dy.cols, at::kFloat, &dw) < 0 ||
      vector(a[7], "dB", dev, true, g.dy.cols, at::kFloat, &db) < 0)
    return nullptr;
  const int hh = view(a[8], "dH", dev, true, &dh);
  if (hh < 0) return nullptr;
  g.dh = hh ? &dh : nullptr;
  g.weight = w;
  g.weight_dtype = wt;
  g.mean = static_cast<const float*>(mean);
  g.rstd = static_cast<const float*>(rstd);
  g.dweight = static_cast<float*>(dw);
  g.dbias = static_cast<float*>(db);
  // the partial sums' memory: the caller's, or this call's own (see rmsnorm_bwd)
  void* wp = nullptr;
  size_t wn = 0;
  at::Tensor own;
  if (a[9] != Py_None) {
    const at::Tensor* ws = tensor(a[9], "workspace", dev);
    if (ws == nullptr) return nullptr;
    wp = ws->data_ptr();
    wn = static_cast<size_t>(ws->numel());
  } else if (dw != nullptr || db != nullptr) {
    wn = size_on(dev, gge_workspace_size_layernorm_bwd, g.dy.cols);
    own = at::empty({static_cast<int64_t>(wn)},
                    at::TensorOptions().dtype(at::kByte).device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)));
    wp = own.data_ptr();
  }
  GGE_CALL(dev, gge_layernorm_bwd(&g, wp, wn, st));
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
                          method<zeroed>("zeroed"), method<b128_wrap>("b128_wrap"),
                          method<b128_quantize>("b128_quantize"), method<b128_transpose>("b128_transpose"),
                          method<b128_dequantize>("b128_dequantize"), method<gemm_b128>("gemm_b128"),
                          method<layernorm>("layernorm"), method<layernorm_bwd>("layernorm_bwd"),
                          {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "gge_marshal", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit_gge_marshal() {
  return PyModule_Create(&kModule);
}
