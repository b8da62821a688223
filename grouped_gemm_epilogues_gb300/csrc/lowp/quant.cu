// Microscaled quantisation and its inverse.
//
// The blocks of a quantised matrix run along its columns (a product's K).  The
// source may hold those contiguously (stride_col 1) or be the transpose of a
// row-major matrix (stride_row 1), as the weight-gradient products need it: a
// tile then goes through shared memory.  Both forms read the source once and
// are bound by memory.
#include "../gge_ptx.cuh"
#include "lowp_launch.h"
#include "mx_format.cuh"

namespace gge {
namespace lowp {
namespace {

using namespace mx;

__device__ __forceinline__ QuantOut quant_out(const QuantPtrs& q, int64_t batch) {
  const int vs = q.v_dtype == 4 ? 4 : 2;
  return QuantOut{q.codes + batch * q.batch_stride, q.ld, q.scales + batch * q.scale_batch_stride,
                  q.kgroups, q.tensor_scale,
                  q.values == nullptr
                      ? nullptr
                      : static_cast<void*>(static_cast<uint8_t*>(q.values) + batch * q.values_batch_stride * vs),
                  q.ldv, q.v_dtype, q.v_vec};
}

// Columns contiguous: a lane takes eight of them, and the lanes of one scale
// word (16, or 8 for nvfp4) stay in one row; words are numbered row by row.
template <typename T, int FMT>
__global__ void quantize_rows_kernel(const __grid_constant__ QuantParams p) {
  constexpr int kLanes = Fmt<FMT>::kGroup / 8;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t batch = blockIdx.y;
  const QuantOut q = quant_out(p.q, batch);
  const T* x = static_cast<const T*>(p.x) + batch * p.stride_batch;
  const float tscale = (FMT == FMT_NVFP4 && q.tensor_scale) ? *q.tensor_scale : 1.f;
  const int64_t words = p.rows * q.kgroups;
  const int64_t per_block = blockDim.x / kLanes;
  const int32_t cols = static_cast<int32_t>(p.cols);
  for (int64_t w0 = blockIdx.x * per_block; w0 < words; w0 += gridDim.x * per_block) {
    const int64_t w = w0 + threadIdx.x / kLanes;
    const bool live = w < words;
    const int64_t row = live ? w / q.kgroups : 0;
    const int32_t col = static_cast<int32_t>(live ? w - row * q.kgroups : 0) * Fmt<FMT>::kGroup +
                        static_cast<int32_t>(threadIdx.x % kLanes) * 8;
    float v[8];
    const T* src = x + row * p.stride_row + col;
    if (live && p.vec && col + 8 <= cols) {
      widen(load8(src), v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = live && col + i < cols ? to_float<T>(src[i]) : 0.f;
    }
    quantise_chunk<FMT>(q, v, row, col, cols, tscale, live);
  }
}

// Rows contiguous (the transpose of a row-major source): a block takes 64 rows x
// 128 columns, reads source lines of 64 values, and each thread quantises 8
// columns of one row out of shared memory.
constexpr int kTRows = 64, kTCols = 128;

template <typename T, int FMT>
__global__ void __launch_bounds__(256) quantize_cols_kernel(const __grid_constant__ QuantParams p) {
  __shared__ T tile[kTCols][kTRows + 4 / sizeof(T)];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t batch = blockIdx.z;
  const QuantOut q = quant_out(p.q, batch);
  const T* x = static_cast<const T*>(p.x) + batch * p.stride_batch;
  const float tscale = (FMT == FMT_NVFP4 && q.tensor_scale) ? *q.tensor_scale : 1.f;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kTRows;
  const int32_t cols = static_cast<int32_t>(p.cols);
  const int32_t col0 = blockIdx.y * kTCols;
  const int r = threadIdx.x % kTRows;
  for (int c = threadIdx.x / kTRows; c < kTCols; c += 256 / kTRows) {
    const int32_t col = col0 + c;
    T v = from_float<T>(0.f);
    if (row0 + r < p.rows && col < cols) v = x[col * p.stride_col + row0 + r];
    tile[c][r] = v;
  }
  __syncthreads();
  // 16 consecutive threads take the 16 chunks of a row, so that its codes are
  // written in whole lines
  const int chunk = threadIdx.x % 16;
  for (int rr = threadIdx.x / 16; rr < kTRows; rr += 16) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_float<T>(tile[chunk * 8 + i][rr]);
    const int32_t col = col0 + chunk * 8;
    quantise_chunk<FMT>(q, v, row0 + rr, col, cols, tscale,
                        row0 + rr < p.rows && col < q.kgroups * Fmt<FMT>::kGroup);
  }
}

template <typename T, int FMT>
cudaError_t launch_quantize_t(const QuantParams& p, int sms, cudaStream_t st) {
  if (p.stride_col == 1 || p.cols == 1) {
    constexpr int kLanes = Fmt<FMT>::kGroup / 8;
    const int64_t words = p.rows * p.q.kgroups;
    const int64_t want = (words + 256 / kLanes - 1) / (256 / kLanes);
    const int64_t most = static_cast<int64_t>(sms) * 64;
    return launch_pdl(quantize_rows_kernel<T, FMT>,
                      dim3(static_cast<unsigned>(want < most ? want : most), static_cast<unsigned>(p.batch)),
                      dim3(256), 0, st, p);
  }
  const int64_t span = p.q.kgroups * Fmt<FMT>::kGroup;
  return launch_pdl(quantize_cols_kernel<T, FMT>,
                    dim3(static_cast<unsigned>((p.rows + kTRows - 1) / kTRows),
                         static_cast<unsigned>((span + kTCols - 1) / kTCols),
                         static_cast<unsigned>(p.batch)),
                    dim3(256), 0, st, p);
}

template <typename T>
cudaError_t launch_quantize_f(const QuantParams& p, int sms, cudaStream_t st) {
  switch (p.q.format) {
    case FMT_MXFP8: return launch_quantize_t<T, FMT_MXFP8>(p, sms, st);
    case FMT_MXFP4: return launch_quantize_t<T, FMT_MXFP4>(p, sms, st);
    default: return launch_quantize_t<T, FMT_NVFP4>(p, sms, st);
  }
}

// ------------------------------------------------------------- and back

// Eight columns a thread.
template <int FMT>
__global__ void dequantize_kernel(const __grid_constant__ DequantParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t batch = blockIdx.y;
  const uint8_t* codes = p.codes + batch * p.batch_stride;
  const uint8_t* scales = p.scales + batch * p.scale_batch_stride;
  const float tscale = (FMT == FMT_NVFP4 && p.tensor_scale) ? *p.tensor_scale : 1.f;
  const int64_t chunks = (p.cols + 7) / 8;
  const int64_t total = p.rows * chunks;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = i / chunks, col = (i - row * chunks) * 8;
    const uint8_t* c = codes + row * p.ld + col * Fmt<FMT>::kBits / 8;
    uint2 w = make_uint2(0u, 0u);
    if constexpr (FMT == FMT_MXFP8) w = *reinterpret_cast<const uint2*>(c);
    else w.x = *reinterpret_cast<const uint32_t*>(c);
    const int64_t block = col / Fmt<FMT>::kBlock;
    const float unit = scale_value<FMT>(scales[scale_word(row, block >> 2, p.kgroups) + (block & 3)]);
    float v[8];
    unpack8<FMT>(w, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] *= unit;
      if constexpr (FMT == FMT_NVFP4) v[j] *= tscale;
    }
    const int64_t at = batch * p.y_batch_stride + row * p.ldy + col;
    if (p.vec && col + 8 <= p.cols) {
      store8_any(p.y, at, p.dtype, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < p.cols) store_any(p.y, at + j, p.dtype, v[j]);
    }
  }
}

}  // namespace

cudaError_t launch_quantize(const QuantParams& p, int sms, cudaStream_t st) {
  if (p.dtype == 0) return launch_quantize_f<__nv_bfloat16>(p, sms, st);
  if (p.dtype == 1) return launch_quantize_f<__half>(p, sms, st);
  return launch_quantize_f<float>(p, sms, st);
}

cudaError_t launch_dequantize(const DequantParams& p, int sms, cudaStream_t st) {
  const int64_t want = (p.rows * ((p.cols + 7) / 8) + 255) / 256;
  const int64_t most = static_cast<int64_t>(sms) * 64;
  const dim3 grid(static_cast<unsigned>(want < most ? want : most), static_cast<unsigned>(p.batch));
  switch (p.format) {
    case FMT_MXFP8: return launch_pdl(dequantize_kernel<FMT_MXFP8>, grid, dim3(256), 0, st, p);
    case FMT_MXFP4: return launch_pdl(dequantize_kernel<FMT_MXFP4>, grid, dim3(256), 0, st, p);
    default: return launch_pdl(dequantize_kernel<FMT_NVFP4>, grid, dim3(256), 0, st, p);
  }
}

}  // namespace lowp
}  // namespace gge
