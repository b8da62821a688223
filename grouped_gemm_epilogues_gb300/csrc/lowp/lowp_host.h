// Checks that the low-precision entry points share.
#pragma once

#include "../gge_host.h"

namespace gge {

// (a warp's and a block's columns past the last one still have to fit 32 bits)
constexpr int64_t kMaxCols = kMaxExtent - 4096;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool is_value_type(int32_t dt) { return dt == GGE_BF16 || dt == GGE_F16 || dt == GGE_F32; }

// A row-major (or, `any_major`, column-major) view of 16- or 32-bit values that
// may start on any element.
inline gge_status check_values(const gge_tensor& t, bool any_major) {
  if (t.reserved != 0) return GGE_ERR_INVALID_ARG;
  if (!is_value_type(t.dtype)) return GGE_ERR_UNSUPPORTED;
  if (t.rows < 0 || t.cols < 0 || t.batch < 1) return GGE_ERR_INVALID_ARG;
  if (t.rows > kMaxExtent || t.cols > kMaxCols || t.batch > 65535) return GGE_ERR_UNSUPPORTED;
  if (t.rows == 0 || t.cols == 0) return GGE_OK;
  if (t.ptr == nullptr) return GGE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(t.ptr) & (elem_bytes(t.dtype) - 1)) != 0) return GGE_ERR_ALIGNMENT;
  if (t.stride_row < 0 || t.stride_col < 0 || t.stride_batch < 0) return GGE_ERR_INVALID_ARG;
  if (t.cols == 1 || t.stride_col == 1) return GGE_OK;
  if (any_major && (t.rows == 1 || t.stride_row == 1)) return GGE_OK;
  return GGE_ERR_UNSUPPORTED;
}

// Rows of an output must not overlap, within a batch or across batches: a batch lies
// behind the one before, or all batches' first rows lie before the second ones.
inline bool rows_apart(const gge_tensor& t) {
  if (t.rows > 1 && t.stride_row < t.cols) return false;
  if (t.batch <= 1 || t.rows == 0 || t.cols == 0) return true;
  if (t.stride_batch >= (t.rows > 1 ? (t.rows - 1) * t.stride_row : 0) + t.cols) return true;
  return t.stride_batch >= t.cols && t.rows > 1 && t.stride_row >= (t.batch - 1) * t.stride_batch + t.cols;
}

inline bool same_shape(const gge_tensor& t, int64_t rows, int64_t cols, int64_t batch) {
  return t.rows == rows && t.cols == cols && t.batch == batch;
}

// Every row (and batch) of the view starts on a 16-byte boundary.
inline bool rows_aligned(const gge_tensor& t) {
  const int es = elem_bytes(t.dtype);
  return aligned16(t.ptr) && (t.rows <= 1 || t.stride_row * es % 16 == 0) &&
         (t.batch <= 1 || t.stride_batch * es % 16 == 0);
}

// Every row of `t` starts as far past a 16-byte boundary as the same row of `x`.
inline bool rows_alike(const gge_tensor& t, const gge_tensor& x) {
  const int64_t es = elem_bytes(x.dtype);
  return ((reinterpret_cast<uintptr_t>(t.ptr) ^ reinterpret_cast<uintptr_t>(x.ptr)) & 15u) == 0 &&
         (t.rows <= 1 || (t.stride_row - x.stride_row) * es % 16 == 0);
}

inline gge_status launched(cudaError_t e) { return e == cudaSuccess ? GGE_OK : GGE_ERR_CUDA; }

}  // namespace gge
