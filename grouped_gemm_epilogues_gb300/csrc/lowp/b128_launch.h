// Kernel parameters and launchers of the operators on 8 bits with a scale for each block of
// 128: quantisation, transposition, layer norm and the product.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "../gge_launch.h"
#include "../gge_params.h"
#include "b128_format.cuh"
#include "lowp_launch.h"

namespace gge {
namespace b128 {

struct QuantParams {
  int64_t rows, cols, batch;      // of the result
  const void* x;
  int32_t dtype;                  // gge_dtype of x; 2 or 3: codes, scaled by `from`
  int64_t stride_row, stride_col, stride_batch;  // elements; one of the first two is 1
  int32_t aligned;                // every line of the source's storage starts on 16 bytes
  View from, q;
  void* values;
  int64_t ldv, v_batch;
  int32_t v_dtype, v_aligned;
};

struct DequantParams {
  int64_t rows, cols, batch;
  View q;
  void* y;
  int64_t ldy, y_batch;
  int32_t dtype, aligned;
};

cudaError_t launch_quantize(const QuantParams& p, cudaStream_t st);
cudaError_t launch_dequantize(const DequantParams& p, cudaStream_t st);

// ------------------------------------------------------------- layer norm

struct LnParams {
  int64_t rows;
  int32_t cols;
  int32_t dtype;  // of x, residual, residual_out and y
  const void *x, *residual;
  void *h, *y;    // residual_out, y (each may be NULL)
  int64_t ldx, ldr, ldh, ldy;
  const void *weight, *bias;  // NULL: 1, 0
  int32_t p_dtype;
  float eps;
  float *mean, *rstd;
  View q, h8;     // codes NULL: not wanted
  void* values;
  int64_t ldv;
  int32_t v_dtype;
  int32_t w_vec;     // weight and bias start on 16-byte boundaries
  int32_t rows_lie;  // lowp::Rows
};

struct LnBwdParams {
  int64_t rows;
  int32_t cols;
  int32_t dtype;  // of dy, h, dh and dx
  const void *dy, *h, *dh;
  View h8;        // codes NULL: h it is
  void* dx;
  int64_t lddy, ldh, lddh, lddx;
  const void* weight;
  int32_t w_dtype;
  const float *mean, *rstd;
  float *dw, *db;   // NULL: not wanted
  float* partials;  // [blocks][2][cols] sums of the blocks' rows
  int32_t w_vec, rows_lie;
};

cudaError_t launch_ln(const LnParams& p, int sms, cudaStream_t st);
int ln_bwd_blocks(int64_t rows, int sms);
cudaError_t launch_ln_bwd(const LnBwdParams& p, int sms, cudaStream_t st);

// ------------------------------------------------------------- the product

// gemm_kernel's parameters and what the block scales and 8-bit outputs add
//
// A stage is a block's rows of A and of B.  Up to 32 rows of A in all (decoding) take no more room
// than that in small tiles, so that more of B is on its way: the MMA reads 128 rows from there all
// the same, and what it makes of others' bytes is not read.  (16 x 8192 x 4096 19.2 -> 14.2 us.)
constexpr int kFewRows = 32;

struct GemmParams {
  Params p;
  View a, b;           // scales of the operands (their codes come through tensor maps)
  View c8, d8, p8;     // 8-bit forms of C, D and PostAct
  int32_t b_rows_one;  // B has a scale a row: one for each of a tile's columns
  int32_t splits;      // CTAs of a cluster that share a tile's K: 1, 2 or 4
  int32_t by_tma;      // 256-wide tiles without a C: bits 0 to 3: D, PostAct, D8, PostAct8 leave by TMA
  int32_t a_rows;      // rows of A in a stage (small tiles): 128, or 32 where there are no more
};

struct GemmMaps {
  CUtensorMap a, b, d, post;
};

// Tile shapes: 256 x 256 on a CTA pair, 128 x 128 and 128 x 64 on one CTA.
// (one translation unit a tile shape)
template <int BN, int CG>
cudaError_t launch_tile(const GemmMaps& maps, const GemmParams& gp, const LaunchShape& shape, cudaStream_t stream);
// Resident CTAs, or clusters of `cluster` CTAs, on the current device, or -1.
template <int BN, int CG>
int units_tile(bool b_rows_one, size_t smem, int cluster);

}  // namespace b128
}  // namespace gge
