// Kernel parameters and launchers of the low-precision operators: RMS norm
// (forward and backward) and microscaled quantisation.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../gge_launch.h"

namespace gge {
namespace lowp {

// A quantised output as the kernels see it (see mx::QuantOut).
struct QuantPtrs {
  int32_t format;  // gge_mx_format, or mx::FMT_NONE
  uint8_t* codes;
  int64_t ld, batch_stride;
  uint8_t* scales;
  int64_t kgroups, scale_batch_stride;
  const float* tensor_scale;
  void* values;
  int64_t ldv, values_batch_stride;
  int32_t v_dtype;
};

// How the rows of a norm's tensors lie in memory.
//   ALIGNED  every row of every tensor starts on a 16-byte boundary;
//   ALIKE    a row starts equally far (`skew` values) past one in every tensor.  The
//            chunks then start on the boundary before the row, chunk 0 with `skew`
//            values that are not the row's.  A row group takes every 8th row (or every
//            16th ...), so that its skew stays the same: the weights' place and dw's
//            are fixed in registers, and nothing is shifted;
//   ANY      chunks start with the row, and rows.cuh shifts what is read and written.
// Codes with scales want chunks that start with the row (their blocks do), so ALIKE is
// for outputs in values only.
enum Rows { ROWS_ANY = 0, ROWS_ALIGNED = 1, ROWS_ALIKE = 2 };

struct NormParams {
  int64_t rows;
  int32_t cols;
  int32_t dtype;  // of x, residual, residual_out and y
  const void *x, *residual;
  void *h, *y;  // residual_out, y (each may be NULL)
  int64_t ldx, ldr, ldh, ldy;
  const void* weight;
  int32_t w_dtype;
  float eps;
  float* inv;  // NULL: not wanted
  QuantPtrs q;
  int32_t w_vec;     // the weight starts on a 16-byte boundary
  int32_t rows_lie;  // Rows
};

struct NormBwdParams {
  int64_t rows;
  int32_t cols;
  int32_t dtype;  // of dy, h, dh and dx
  const void *dy, *h, *dh;
  void* dx;
  int64_t lddy, ldh, lddh, lddx;
  const void* weight;
  int32_t w_dtype;
  const float* inv;
  float* dw;        // NULL: not wanted
  float* partials;  // [grid][cols] sums of the blocks' rows
  int32_t w_vec, rows_lie;
};

struct QuantParams {
  int64_t rows, cols;
  int64_t batch;
  int32_t dtype;
  const void* x;
  int64_t stride_row, stride_col, stride_batch;  // elements; one of the first two is 1
  int32_t aligned;  // every row of the source's storage and of the values starts on a 16-byte boundary
  QuantPtrs q;
};

struct DequantParams {
  int64_t rows, cols, batch;
  int32_t format;
  const uint8_t *codes, *scales;
  int64_t ld, batch_stride, kgroups, scale_batch_stride;
  const float* tensor_scale;
  void* y;
  int64_t ldy, y_batch_stride;
  int32_t dtype;
  int32_t aligned;
};

cudaError_t launch_norm(const NormParams& p, int sms, cudaStream_t st);
// Blocks a backward launch uses at most (each leaves `cols` partial sums).
int norm_bwd_blocks(int64_t rows, int sms);
cudaError_t launch_norm_bwd(const NormBwdParams& p, int sms, cudaStream_t st);
cudaError_t launch_quantize(const QuantParams& p, cudaStream_t st);
cudaError_t launch_dequantize(const DequantParams& p, cudaStream_t st);

// Launch with programmatic stream serialisation: the kernel sets up, then waits
// (griddepcontrol.wait) for the stream's previous kernel before it touches
// global memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace lowp
}  // namespace gge
