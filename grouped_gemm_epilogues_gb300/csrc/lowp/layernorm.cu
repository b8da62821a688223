// Layer norm: the value type's choice, and the end of the backward's sums over the rows.
#include "b128_launch.h"
#include "norm_rows.cuh"

namespace gge {
namespace b128 {
namespace {

// dw and db: the partial rows' sums, 32 columns a block, and 32 warps that share the rows,
// joined in a fixed order.
__global__ void __launch_bounds__(1024)
    ln_bwd_sum_kernel(const float* partials, int blocks, int32_t cols, float* dw, float* db) {
  __shared__ float part[32][33];
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* out = blockIdx.y == 0 ? dw : db;
  if (out == nullptr) return;
  const float* from = partials + static_cast<int64_t>(blockIdx.y) * cols;
  const int32_t col = blockIdx.x * 32 + lane;
  ptx::griddep_wait();
  float s = 0.f;
  if (col < cols) {
#pragma unroll 8
    for (int b = warp; b < blocks; b += 32) s += from[static_cast<int64_t>(b) * 2 * cols + col];
  }
  part[warp][lane] = s;
  __syncthreads();
  s = lowp::warp_sum(part[lane][warp]);  // column `warp` of the block
  if (lane == 0 && blockIdx.x * 32 + warp < cols) out[blockIdx.x * 32 + warp] = s;
}

}  // namespace

template <typename T>
cudaError_t launch_ln_f(const LnParams& p, int sms, cudaStream_t st);
template <typename T>
cudaError_t launch_ln_bwd_t(const LnBwdParams& p, int sms, cudaStream_t st);

cudaError_t launch_ln_bwd_sum(const LnBwdParams& p, int blocks, cudaStream_t st) {
  return lowp::launch_pdl(ln_bwd_sum_kernel, dim3((p.cols + 31) / 32, 2), dim3(1024), 0, st,
                          static_cast<const float*>(p.partials), blocks, p.cols, p.dw, p.db);
}

cudaError_t launch_ln(const LnParams& p, int sms, cudaStream_t st) {
  if (p.dtype == 0) return launch_ln_f<__nv_bfloat16>(p, sms, st);
  if (p.dtype == 1) return launch_ln_f<__half>(p, sms, st);
  return launch_ln_f<float>(p, sms, st);
}

int ln_bwd_blocks(int64_t rows, int sms) { return static_cast<int>(rows < sms ? rows : sms); }

cudaError_t launch_ln_bwd(const LnBwdParams& p, int sms, cudaStream_t st) {
  if (p.dtype == 0) return launch_ln_bwd_t<__nv_bfloat16>(p, sms, st);
  if (p.dtype == 1) return launch_ln_bwd_t<__half>(p, sms, st);
  return launch_ln_bwd_t<float>(p, sms, st);
}

}  // namespace b128
}  // namespace gge
