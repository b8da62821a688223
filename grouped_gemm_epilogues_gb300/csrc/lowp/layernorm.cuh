// Layer norm with the residual's addition, and its backward.
//
//   h = round(x + residual)      mean, var over a row      rstd = 1 / sqrt(var + eps)
//   y = (h - mean) rstd w + b
//
// y leaves in 16 or 32 bits, or as codes with a scale for each 128 columns; h, too, can leave
// in 8 bits, and the backward read it so.  The variance is that of differences from a mean: a
// thread's sums, of its own values, are joined to a warp's and those to the row's by mean and
// squared deviation,
//   M2 = sum over parts of M2_p + n_p (mean_p - mean)^2,
// with the parts' means taken relative to one of them, and once more relative to the result where
// that one lay far from it (see Joined), so that no sum of squares is large against the variance.
// What is left of a mean far from zero is its own rounding in a thread's differences.  (One
// reduction over the warp for both sums; a warp's mean first and then its deviations: 16384 x 8192 to
// codes and values 281 us, so 228.)
//
// Backward, n = (h - mean) rstd, g = dy w, for dh the gradient that reaches h directly:
//   dx = rstd (g - mean(g) - n mean(g n)) + dh    dw = sum over rows of dy n    db = of dy
//
// Both are bound by memory and built as the RMS norm's kernels (norm.cu): rows on their way to
// shared memory by cp.async while a row is reduced in registers and written, so every value is
// read once; a row's lie in memory (Rows) decides whether anything has to be shifted.
#pragma once

#include <type_traits>

#include "b128_launch.h"
#include "norm_rows.cuh"

namespace gge {
namespace b128 {

cudaError_t launch_ln_bwd_sum(const LnBwdParams& p, int blocks, cudaStream_t st);


using namespace mx;
using namespace lowp;

// Eight values of a parameter from column col on; `none` where there is no such parameter.
__device__ __forceinline__ void load_param(const void* w, int32_t dtype, int32_t vec, int32_t col, int32_t cols,
                                           float none, float2 (&v)[4]) {
  if (w != nullptr) {
    load_weight(w, dtype, vec, col, cols, v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(none, none);
  }
}

// Both parameters where all eight values of both are there and aligned: one choice of the type.
// (Outputs in codes, which are bound by instructions: 16384 x 8192 228 -> 212 us.  Outputs in 16 bits
// are not, and lose the registers: 170 -> 212.)
template <typename W>
__device__ __forceinline__ void both_params(const void* w, const void* b, int32_t col, float2 (&v)[4], float2 (&u)[4]) {
  const Raw8<W> rw = load8(static_cast<const W*>(w) + col), rb = load8(static_cast<const W*>(b) + col);
  widen(rw, v);
  widen(rb, u);
}

__device__ __forceinline__ float2 add2(float2 a, float b) { return __fadd2_rn(a, make_float2(b, b)); }
__device__ __forceinline__ float2 mul2(float2 a, float b) { return __fmul2_rn(a, make_float2(b, b)); }

// Two sums over the `tpr` threads that share a row (see row_sum).
__device__ __forceinline__ float2 row_sum2(float a, float b, int tpr, float2* slots, int flip, int sub) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (tpr == 32) return make_float2(a, b);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = tpr >> 5;
  float2* s = slots + flip * 32;
  if (lane == 0) s[warp] = make_float2(a, b);
  asm volatile("bar.sync %0, %1;" ::"r"(sub + 1), "r"(tpr) : "memory");
  const float2 v = lane < per ? s[sub * per + lane] : make_float2(0.f, 0.f);
  return make_float2(warp_sum(v.x), warp_sum(v.y));
}

__device__ __forceinline__ void warp_sums(float& a, float& b) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
}

// Parts of a row joined: with off = mean_p - pivot, total = sum n_p off and square = sum (M2_p + n_p off^2),
//   mean = pivot + total / n      M2 = square - total^2 / n.
// The difference loses as much as square is larger than M2: where the pivot, one of the parts' means,
// is that of a part with a value far from all others, 32 times and more.  `far`: then it has to be
// done again relative to the mean just found.  (With M2 above two thirds of square a join keeps 24
// units: three roundings and five additions of up to 1.5 M2, and seven of total, up to sqrt(0.75) M2.)
struct Joined {
  float mean, m2;
  bool far;
};
__device__ __forceinline__ Joined joined(float pivot, float total, float square, float inv_n) {
  const float d = total * inv_n, m2 = fmaf(-total, d, square);
  // (rounding may have left M2 below zero; a NaN stays one, as of a row that holds an infinity or a
  // NaN nothing is a number)
  return Joined{pivot + d, m2 < 0.f ? 0.f : m2, square > 1.5f * m2};
}

// Columns of [col, col + n) that a row of `cols` has.
__device__ __forceinline__ int32_t columns_in(int32_t col, int32_t n, int32_t cols) {
  return max(min(col + n, cols) - max(col, 0), 0);
}

// Quantise a lane's eight values (warp-collective) and store codes and scale; the numbers that
// the codes stand for come back in v.
__device__ __forceinline__ void put_codes(const View& q, uint32_t row, int32_t col, int32_t cols, float2 (&v)[4],
                                          bool back) {
  float unit;
  const uint2 z = q.e5m2 ? quantise8<true>(v, unit) : quantise8<false>(v, unit);
  // (one row a block)
  if ((threadIdx.x & 15) == 0 && col < cols) q.scales[row * q.s_row + static_cast<uint32_t>(col >> 7) * q.s_col] = unit;
  store_codes8(q.codes + row * q.ld + col, z, cols - col);
  if (back) values8_any(q.e5m2 != 0, z, unit, v);
}

// ------------------------------------------------------------ forward

// Threads a block has at most, and rows in shared memory: as in the RMS norm.
template <int R>
constexpr int ln_threads() {
  return R == ROWS_ALIKE ? kRowThreads : kMaxThreads;
}
template <typename T, int C, int R>
constexpr int ln_depth() {
  return ring_depth(ln_threads<R>() / 32 * C * 2 * WarpRow<T>::kBytes, R == ROWS_ALIKE ? 4 : 2);
}

// A row is spread over `tpr` threads; thread i holds the 8-value chunks i, i + tpr, ...
template <typename T, int C, bool CODES, int R>
__global__ void __launch_bounds__(ln_threads<R>()) ln_kernel(const __grid_constant__ LnParams p, int tpr) {
  __shared__ float2 slots[64];
  __shared__ float counts[32];
  extern __shared__ uint8_t ring_raw[];
  ptx::griddep_launch_dependents();
  const int per_block = blockDim.x / tpr;
  const int sub = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int32_t cols = p.cols;
  constexpr int D = ln_depth<T, C, R>();
  const bool has_res = p.residual != nullptr;
  const bool whole_params = CODES && p.weight != nullptr && p.bias != nullptr && p.w_vec != 0;
  // this warp's buffers: [row in flight][chunk][x, residual]
  constexpr uint32_t kBuf = WarpRow<T>::kBytes;
  constexpr uint32_t kRow = 2 * C * kBuf;
  const uint32_t ring = ptx::smem_addr(ring_raw) + warp * kRow;
  const uint32_t ring_row = warps * kRow;
  const uint32_t rows = static_cast<uint32_t>(p.rows);  // (below 2^31, and so is a step past them)
  const uint32_t step = gridDim.x * per_block;
  uint32_t row = blockIdx.x * per_block + sub;
  RowReader<T, R> x, res;
  const int32_t skew = R == ROWS_ALIKE ? row_skew<T>(static_cast<const T*>(p.x) + row * p.ldx) : 0;
  const int32_t col0 = t * 8 - skew;         // chunk 0's first column
  const int32_t warp_col = col0 - lane * 8;  // and its warp's
  x.init(p.x, p.ldx, row, col0);
  res.init(p.residual, p.ldr, row, col0);
  // columns that this warp holds
  int32_t n_warp = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) n_warp += columns_in(warp_col + c * tpr * 8, 256, cols);
  const float n_mine = static_cast<float>(n_warp);
  int32_t n_own = 0;  // and this thread
#pragma unroll
  for (int c = 0; c < C; ++c) n_own += columns_in(col0 + c * tpr * 8, 8, cols);
  const float n_thread = static_cast<float>(n_own), inv_thread = n_own > 0 ? 1.f / n_thread : 0.f;
  const float inv_mine = n_warp > 0 ? 1.f / n_mine : 0.f;
  if (lane == 0) counts[warp] = n_mine;
  __syncthreads();
  const int per = tpr >> 5;
  const float n_lane = lane < per ? counts[sub * per + lane] : 0.f;  // of the row's warp `lane`
  ptx::griddep_wait();
#pragma unroll
  for (int s = 0; s < D * C * 2; ++s)
    RowReader<T, R>::clear(ring + s / (C * 2) * ring_row + s % (C * 2) * kBuf, col0 + s % (C * 2) / 2 * tpr * 8, cols);
  constexpr bool kHeld = R == ROWS_ALIKE;  // weight and bias stay in registers
  float2 wk[kHeld ? C : 1][4], bk[kHeld ? C : 1][4];
  if constexpr (kHeld) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      load_param(p.weight, p.p_dtype, 0, col0 + c * tpr * 8, cols, 1.f, wk[c]);
      load_param(p.bias, p.p_dtype, 0, col0 + c * tpr * 8, cols, 0.f, bk[c]);
    }
  }
  uint32_t ahead = row;
  const auto start = [&](int slot) {
    if (ahead < rows) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t dst = ring + slot * ring_row + c * 2 * kBuf;
        const int32_t over = c * tpr * 8;
        x.copy(dst, col0 + over, c, over, cols, ahead * p.ldx < 8);
        if (has_res) res.copy(dst + kBuf, col0 + over, c, over, cols, ahead * p.ldr < 8);
      }
      x.next += static_cast<int64_t>(step) * p.ldx;
      res.next += static_cast<int64_t>(step) * p.ldr;
    }
    ahead += step;
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s + 1 < D; ++s) start(s);
  const float inv_cols = 1.f / static_cast<float>(cols);
  int slot = 0, flip = 0;
  // (Made twice, with a residual and without: one loop that asks each time is too much for the compiler
  // to take apart by itself, and costs 16384 x 8192 in 16 bits 158 us for 133, 211 for 176 with a residual.)
  const auto all_rows = [&](auto with_residual) {
    constexpr bool kRes = decltype(with_residual)::value;
    for (; row < rows; row += step) {
      if constexpr (R == ROWS_ANY) __syncwarp();  // (the slot was read in the iteration before)
      start((slot + D - 1) % D);
      cp_async_wait<D - 1>();
      if constexpr (R == ROWS_ANY) __syncwarp();
      Raw8<T> h[C];
      float2 sum = make_float2(0.f, 0.f), v[C][4];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int32_t col = col0 + c * tpr * 8;
        const uint32_t src = ring + slot * ring_row + c * 2 * kBuf;
        h[c] = take_chunk<T, R>(src, c, static_cast<const T*>(p.x) + row * p.ldx, col, cols);
        if constexpr (kRes) {
          h[c] = add8(h[c], take_chunk<T, R>(src + kBuf, c, static_cast<const T*>(p.residual) + row * p.ldr, col, cols));
          if (p.h != nullptr && warp_col + c * tpr * 8 < cols)
            put_chunk<T, R>(static_cast<T*>(p.h) + row * p.ldh, c, col, cols, h[c]);
        }
        widen(h[c], v[c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = __fadd2_rn(sum, v[c][i]);
      }
      slot = (slot + 1) % D;
      // a thread's mean and squared deviation, joined over the warp as the warps' are over the row
      const float own = (sum.x + sum.y) * inv_thread;
      float2 dev = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int32_t col = col0 + c * tpr * 8;
        if (col >= 0 && col + 8 <= cols) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 d = add2(v[c][i], -own);
            dev = __ffma2_rn(d, d, dev);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int32_t a = col + 2 * i, b = a + 1;
            const float2 d = make_float2(a >= 0 && a < cols ? v[c][i].x - own : 0.f, b >= 0 && b < cols ? v[c][i].y - own : 0.f);
            dev = __ffma2_rn(d, d, dev);
          }
        }
      }
      // (relative to the second thread's: of a row that starts elsewhere the first may hold one value.
      // Both sums are the same bits in every lane, so `far` is the warp's)
      Joined all;
      const auto join_threads = [&](float pivot) {
        const float off = own - pivot;
        float total = n_thread * off, square = fmaf(total, off, dev.x + dev.y);
        warp_sums(total, square);
        all = joined(pivot, total, square, inv_mine);
      };
      join_threads(__shfl_sync(0xffffffffu, own, 1));
      if (__builtin_expect(all.far, 0)) join_threads(all.mean);
      if (tpr > 32) {
        float2* at = slots + flip * 32;
        if (lane == 0) at[warp] = make_float2(all.mean, all.m2);
        asm volatile("bar.sync %0, %1;" ::"r"(sub + 1), "r"(tpr) : "memory");
        const float2 w = lane < per ? at[sub * per + lane] : make_float2(0.f, 0.f);
        const auto join_warps = [&](float pivot) {
          const float off = w.x - pivot;
          float total = n_lane * off, square = fmaf(total, off, w.y);
          warp_sums(total, square);
          all = joined(pivot, total, square, inv_cols);
        };
        join_warps(__shfl_sync(0xffffffffu, w.x, 0));
        if (__builtin_expect(all.far, 0)) join_warps(all.mean);
        flip ^= 1;
      }
      const float mean = all.mean;
      // (rounded correctly: an error of rstd moves every value of the row the same way)
      const float rstd = __frsqrt_rn(fmaf(all.m2, inv_cols, p.eps));
      if (t == 0) {
        if (p.mean != nullptr) p.mean[row] = mean;
        if (p.rstd != nullptr) p.rstd[row] = rstd;
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int32_t col = col0 + c * tpr * 8;
        if (c > 0 && warp_col + c * tpr * 8 >= cols) continue;
        float2 v[4], w[4], b[4];
        widen(h[c], v);
        if constexpr (CODES) {
          if (p.h8.codes != nullptr) {
            float2 u[4] = {v[0], v[1], v[2], v[3]};
            put_codes(p.h8, row, col, cols, u, false);
          }
        }
        if constexpr (!kHeld) {
          if (whole_params && col + 8 <= cols) {
            if (p.p_dtype == DT_BF16) both_params<__nv_bfloat16>(p.weight, p.bias, col, w, b);
            else if (p.p_dtype == DT_F16) both_params<__half>(p.weight, p.bias, col, w, b);
            else both_params<float>(p.weight, p.bias, col, w, b);
          } else {
            load_param(p.weight, p.p_dtype, p.w_vec, col, cols, 1.f, w);
            load_param(p.bias, p.p_dtype, p.w_vec, col, cols, 0.f, b);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = __ffma2_rn(mul2(add2(v[i], -mean), rstd), kHeld ? wk[kHeld ? c : 0][i] : w[i], kHeld ? bk[kHeld ? c : 0][i] : b[i]);
        if (p.y != nullptr) put_chunk<T, R>(static_cast<T*>(p.y) + row * p.ldy, c, col, cols, narrow<T>(v));
        if constexpr (CODES) {
          if (p.q.codes != nullptr) {
            // (past the row's end the values are -mean rstd, not 0)
            if (col + 8 > cols) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (col + 2 * i >= cols) v[i].x = 0.f;
                if (col + 2 * i + 1 >= cols) v[i].y = 0.f;
              }
            }
            put_codes(p.q, row, col, cols, v, p.values != nullptr);
            if (p.values != nullptr)
              store_row8_any<R == ROWS_ALIGNED>(p.values, row * p.ldv, p.v_dtype, col, cols, v);
          }
        }
      }
    }
  };
  if (has_res) all_rows(std::true_type{});
  else all_rows(std::false_type{});
}

// Sum over a whole block.
__device__ __forceinline__ float block_sum(float v, float* slots, int& flip) {
  const float s = row_sum(v, blockDim.x, slots, flip, 0);
  flip ^= 1;
  return s;
}

// Rows too long for a block's registers: four values a lane, 128 columns a warp, and two more
// passes that read the row again (from L2).
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) ln_long_kernel(const __grid_constant__ LnParams p) {
  __shared__ float slots[64];
  ptx::griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t cols = p.cols;
  ptx::griddep_wait();
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* res = p.residual != nullptr ? static_cast<const T*>(p.residual) + row * p.ldr : nullptr;
    const auto value = [&](int32_t col) {
      const float a = to_float<T>(x[col]);
      return res != nullptr ? to_float<T>(from_float<T>(a + to_float<T>(res[col]))) : a;
    };
    float s = 0.f;
#pragma unroll 4
    for (int32_t col = threadIdx.x; col < cols; col += kMaxThreads) s += value(col);
    const float mean = block_sum(s, slots, flip) / static_cast<float>(cols);
    s = 0.f;
#pragma unroll 4
    for (int32_t col = threadIdx.x; col < cols; col += kMaxThreads) {
      const float d = value(col) - mean;
      s = fmaf(d, d, s);
    }
    const float rstd = __frsqrt_rn(block_sum(s, slots, flip) / static_cast<float>(cols) + p.eps);
    if (threadIdx.x == 0) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    for (int32_t first = warp * 128; first < cols; first += kMaxThreads * 4) {  // (the whole warp)
      float h[4], y[4];
      uint32_t top_h = 0u, top_y = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t col = first + lane * 4 + i;
        h[i] = y[i] = 0.f;
        if (col < cols) {
          h[i] = value(col);
          const float w = p.weight != nullptr ? load_any(p.weight, col, p.p_dtype) : 1.f;
          const float b = p.bias != nullptr ? load_any(p.bias, col, p.p_dtype) : 0.f;
          y[i] = fmaf((h[i] - mean) * rstd, w, b);
        }
        top_h = max(top_h, abs_bits(h[i]));
        top_y = max(top_y, abs_bits(y[i]));
      }
      const auto codes = [&](const View& q, const float (&v)[4], uint32_t top, float (&back)[4]) {
        top = __reduce_max_sync(0xffffffffu, top);
        float factor;
        const float unit = q.e5m2 ? block_scale<true>(top, factor) : block_scale<false>(top, factor);
        const uint32_t z = q.e5m2 ? pack4<true>(v[0] * factor, v[1] * factor, v[2] * factor, v[3] * factor)
                                  : pack4<false>(v[0] * factor, v[1] * factor, v[2] * factor, v[3] * factor);
        if (lane == 0) *q.scale(row, first >> 7, 0) = unit;
        uint8_t* at = q.codes + row * q.ld + first + lane * 4;
        const int32_t n = cols - first - lane * 4;
        if (n >= 4) {
          *reinterpret_cast<uint32_t*>(at) = z;
        } else {
#pragma unroll
          for (int i = 0; i < 3; ++i)
            if (i < n) at[i] = static_cast<uint8_t>(z >> (8 * i));
        }
        float2 b[2];
        if (q.e5m2) values4<true>(z, unit, b);
        else values4<false>(z, unit, b);
        back[0] = b[0].x, back[1] = b[0].y, back[2] = b[1].x, back[3] = b[1].y;
      };
      float back[4];
      if (p.h8.codes != nullptr) codes(p.h8, h, top_h, back);
      if (p.q.codes != nullptr) codes(p.q, y, top_y, back);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t col = first + lane * 4 + i;
        if (col >= cols) break;
        if (res != nullptr && p.h != nullptr) static_cast<T*>(p.h)[row * p.ldh + col] = from_float<T>(h[i]);
        if (p.y != nullptr) static_cast<T*>(p.y)[row * p.ldy + col] = from_float<T>(y[i]);
        if (p.values != nullptr) store_any(p.values, row * p.ldv + col, p.v_dtype, back[i]);
      }
    }
  }
}

template <typename T, int C, bool CODES, int R>
cudaError_t launch_ln_c(const LnParams& p, const RowShape& s, int sms, cudaStream_t st) {
  const int block = s.per * s.tpr;
  const size_t smem = static_cast<size_t>(ln_depth<T, C, R>()) * (block / 32) * C * 2 * WarpRow<T>::kBytes;
  const cudaError_t e = allow_smem<ln_kernel<T, C, CODES, R>>();
  if (e != cudaSuccess) return e;
  // as many blocks as an SM holds, each with its share of the rows
  const int64_t resident = static_cast<int64_t>(sms) * s.blocks;
  const int64_t want = (p.rows + s.per - 1) / s.per;
  int blocks = static_cast<int>(want < resident ? want : resident);
  if (R == ROWS_ALIKE) blocks = alike_blocks(p.rows, s.per, blocks);
  return launch_pdl(ln_kernel<T, C, CODES, R>, dim3(blocks), dim3(block), smem, st, p, s.tpr);
}

template <typename T, bool CODES>
cudaError_t launch_ln_t(const LnParams& p, int sms, cudaStream_t st) {
  if (p.cols <= kMaxCols) {
    if constexpr (!CODES) {
      const int64_t chunks = alike_chunks(p.cols, sizeof(T));
      if (p.rows_lie == ROWS_ALIKE && chunks * 8 <= kMaxCols && sms >= 8) {
        const RowShape s = many_registers(chunks, sizeof(T) == 2 ? 64 : 2 * kRowThreads, p.rows, sms);
        return s.c == 1   ? launch_ln_c<T, 1, CODES, ROWS_ALIKE>(p, s, sms, st)
               : s.c == 2 ? launch_ln_c<T, 2, CODES, ROWS_ALIKE>(p, s, sms, st)
                          : launch_ln_c<T, 4, CODES, ROWS_ALIKE>(p, s, sms, st);
      }
    }
    const RowShape s = many_threads((p.cols + 7) / 8, p.rows <= sms);
    if (p.rows_lie == ROWS_ALIGNED)
      return s.c == 1 ? launch_ln_c<T, 1, CODES, ROWS_ALIGNED>(p, s, sms, st)
                      : launch_ln_c<T, 2, CODES, ROWS_ALIGNED>(p, s, sms, st);
    return s.c == 1 ? launch_ln_c<T, 1, CODES, ROWS_ANY>(p, s, sms, st)
                    : launch_ln_c<T, 2, CODES, ROWS_ANY>(p, s, sms, st);
  }
  return launch_pdl(ln_long_kernel<T>, dim3(static_cast<unsigned>(p.rows < 65536 ? p.rows : 65536)), dim3(kMaxThreads),
                    0, st, p);
}

template <typename T>
cudaError_t launch_ln_f(const LnParams& p, int sms, cudaStream_t st) {
  return p.q.codes != nullptr || p.h8.codes != nullptr ? launch_ln_t<T, true>(p, sms, st)
                                                       : launch_ln_t<T, false>(p, sms, st);
}

// ----------------------------------------------------------- backward

template <typename T, int C, int R>
constexpr int bwd_depth() {
  return ring_depth(kRowThreads / 32 * C * 3 * WarpRow<T>::kBytes, R == ROWS_ALIKE ? 4 : 3);
}

// 8 codes a lane on their way to shared memory; codes past the row's end arrive as zeros.
__device__ __forceinline__ void copy_codes(uint32_t dst, const uint8_t* at, int32_t left) {
  if (left > 0)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst + (threadIdx.x & 31) * 8), "l"(at),
                 "r"(min(8, left))
                 : "memory");
}

// A block takes as many rows at a time as its threads hold.  Each thread keeps its columns'
// share of dw and db in registers; at the end the block's row groups add theirs up and leave
// one row of partial sums each.  H8: h comes as codes.
template <typename T, int C, int R, bool H8>
__global__ void __launch_bounds__(kRowThreads) ln_bwd_kernel(const __grid_constant__ LnBwdParams p, int tpr) {
  __shared__ float2 slots[64];
  extern __shared__ uint8_t ring_raw[];
  ptx::griddep_launch_dependents();
  // g and n stay in registers over the row's sums, or are made again from shared memory; so do
  // the weights, or they are read again
  constexpr bool kKeep = C < 4;
  const int per_block = blockDim.x / tpr;
  const int sub = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int lane = threadIdx.x & 31;
  const int32_t cols = p.cols;
  constexpr uint32_t kBuf = WarpRow<T>::kBytes;
  constexpr int D = bwd_depth<T, C, R>();
  const bool has_dh = p.dh != nullptr;
  // this warp's buffers: [row in flight][chunk][dy, h, dh]
  constexpr uint32_t kRow = 3 * C * kBuf;
  const uint32_t ring = ptx::smem_addr(ring_raw) + (threadIdx.x >> 5) * kRow;
  const uint32_t ring_row = (blockDim.x >> 5) * kRow;
  const uint32_t rows = static_cast<uint32_t>(p.rows);  // (below 2^31, and so is a step past them)
  const uint32_t step = gridDim.x * per_block;
  uint32_t row = blockIdx.x * per_block + sub;
  RowReader<T, R> dy, h, dh;
  const int32_t skew = R == ROWS_ALIKE ? row_skew<T>(static_cast<const T*>(p.dy) + row * p.lddy) : 0;
  const int32_t col0 = t * 8 - skew;         // chunk 0's first column
  const int32_t warp_col = col0 - lane * 8;  // and its warp's
  dy.init(p.dy, p.lddy, row, col0);
  if constexpr (!H8) h.init(p.h, p.ldh, row, col0);
  dh.init(p.dh, p.lddh, row, col0);
  ptx::griddep_wait();
  float2 dw[C][4], db[C][4], w[kKeep ? C : 1][4];
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[c][i] = db[c][i] = make_float2(0.f, 0.f);
    if constexpr (kKeep) load_param(p.weight, p.w_dtype, R == ROWS_ALIKE ? 0 : p.w_vec, col0 + c * tpr * 8, cols, 1.f, w[c]);
  }
#pragma unroll
  for (int s = 0; s < D * C * 3; ++s)
    RowReader<T, R>::clear(ring + s / (C * 3) * ring_row + s % (C * 3) * kBuf, col0 + s % (C * 3) / 3 * tpr * 8, cols);
  uint32_t ahead = row;
  const auto start = [&](int slot) {
    if (ahead < rows) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t dst = ring + slot * ring_row + c * 3 * kBuf;
        const int32_t over = c * tpr * 8, col = col0 + over;
        dy.copy(dst, col, c, over, cols, ahead * p.lddy < 8);
        if constexpr (H8) copy_codes(dst + kBuf, p.h8.codes + ahead * p.h8.ld + col, cols - col);
        else h.copy(dst + kBuf, col, c, over, cols, ahead * p.ldh < 8);
        if (has_dh) dh.copy(dst + 2 * kBuf, col, c, over, cols, ahead * p.lddh < 8);
      }
      dy.next += static_cast<int64_t>(step) * p.lddy;
      if constexpr (!H8) h.next += static_cast<int64_t>(step) * p.ldh;
      dh.next += static_cast<int64_t>(step) * p.lddh;
    }
    ahead += step;
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s + 1 < D; ++s) start(s);
  const float inv_cols = 1.f / static_cast<float>(cols);
  int slot = 0, flip = 0;
  // a row's scalars are fetched a row ahead
  float mean_next = 0.f, rstd_next = 0.f, unit_next[H8 ? C : 1];
  const auto fetch = [&](uint32_t at) {
    if (at >= rows) return;
    mean_next = p.mean[at];
    rstd_next = p.rstd[at];
    if constexpr (H8) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int32_t col = col0 + c * tpr * 8;
        unit_next[c] = col < cols ? *p.h8.scale(at, col >> 7, 0) : 0.f;
      }
    }
  };
  fetch(row);
  for (; row < rows; row += step) {
    if constexpr (R == ROWS_ANY) __syncwarp();
    start((slot + D - 1) % D);
    const float mean = mean_next, rstd = rstd_next;
    float unit[H8 ? C : 1];
    if constexpr (H8) {
#pragma unroll
      for (int c = 0; c < C; ++c) unit[c] = unit_next[c];
    }
    fetch(row + step);
    cp_async_wait<D - 1>();
    if constexpr (R == ROWS_ANY) __syncwarp();
    const uint32_t src = ring + slot * ring_row;
    // dy w and n of chunk c (g holds dy where `raw`)
    const auto take = [&](int c, float2 (&z)[4], float2 (&n)[4]) {
      const int32_t col = col0 + c * tpr * 8;
      widen(take_chunk<T, R>(src + c * 3 * kBuf, c, static_cast<const T*>(p.dy) + row * p.lddy, col, cols), z);
      if constexpr (H8) {
        uint2 k = make_uint2(0u, 0u);
        if (col < cols) {
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(k.x), "=r"(k.y) : "r"(src + c * 3 * kBuf + kBuf + lane * 8) : "memory");
        }
        values8_any(p.h8.e5m2 != 0, k, unit[H8 ? c : 0], n);
      } else {
        widen(take_chunk<T, R>(src + c * 3 * kBuf + kBuf, c, static_cast<const T*>(p.h) + row * p.ldh, col, cols), n);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) n[i] = mul2(add2(n[i], -mean), rstd);
    };
    const auto weights = [&](int c, float2 (&u)[4]) {
      if constexpr (kKeep) {
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = w[kKeep ? c : 0][i];
      } else {
        load_param(p.weight, p.w_dtype, R == ROWS_ALIKE ? 0 : p.w_vec, col0 + c * tpr * 8, cols, 1.f, u);
      }
    };
    float2 g[kKeep ? C : 1][4], n[kKeep ? C : 1][4];
    float2 a = make_float2(0.f, 0.f), b = a;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float2(&z)[4] = g[kKeep ? c : 0];
      float2(&m)[4] = n[kKeep ? c : 0];
      float2 u[4];
      take(c, z, m);
      weights(c, u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // (z is zero outside the row, where m is not)
        dw[c][i] = __ffma2_rn(z[i], m[i], dw[c][i]);
        db[c][i] = __fadd2_rn(z[i], db[c][i]);
        z[i] = __fmul2_rn(z[i], u[i]);
        a = __fadd2_rn(z[i], a);
        b = __ffma2_rn(z[i], m[i], b);
      }
    }
    const float2 sums = row_sum2(a.x + a.y, b.x + b.y, tpr, slots, flip, sub);
    flip ^= 1;
    const float ka = -sums.x * inv_cols, kb = -sums.y * inv_cols;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int32_t col = col0 + c * tpr * 8;
      if (warp_col + c * tpr * 8 >= cols) continue;
      float2(&z)[4] = g[kKeep ? c : 0];
      float2(&m)[4] = n[kKeep ? c : 0];
      if constexpr (!kKeep) {
        float2 u[4];
        take(c, z, m);
        weights(c, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = __fmul2_rn(z[i], u[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = mul2(__ffma2_rn(m[i], make_float2(kb, kb), add2(z[i], ka)), rstd);
      if (has_dh) {
        float2 v[4];
        widen(take_chunk<T, R>(src + c * 3 * kBuf + 2 * kBuf, c, static_cast<const T*>(p.dh) + row * p.lddh, col, cols), v);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = __fadd2_rn(z[i], v[i]);
      }
      put_chunk<T, R>(static_cast<T*>(p.dx) + row * p.lddx, c, col, cols, narrow<T>(z));
    }
    slot = (slot + 1) % D;
  }
  if (p.partials == nullptr) return;
  // the row groups' sums, added in their order: dw's, then db's
  cp_async_wait<0>();
  float* sums = reinterpret_cast<float*>(ring_raw);  // [group][8 + column]
  const int32_t pitch = tpr * C * 8 + 8;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float* at = sums + sub * pitch + 8 + col0 + c * tpr * 8 + 2 * i;
        const float2 v = k == 0 ? dw[c][i] : db[c][i];
        if constexpr (R == ROWS_ALIKE) at[0] = v.x, at[1] = v.y;
        else *reinterpret_cast<float2*>(at) = v;
      }
    __syncthreads();
    for (int32_t col = threadIdx.x; col < cols; col += blockDim.x) {
      float s = 0.f;
      for (int i = 0; i < per_block; ++i) s += sums[i * pitch + 8 + col];
      p.partials[(static_cast<int64_t>(blockIdx.x) * 2 + k) * cols + col] = s;
    }
  }
}

// h of one place, from either form.
template <typename T>
__device__ __forceinline__ float h_at(const LnBwdParams& p, int64_t row, int32_t col) {
  if (p.h8.codes == nullptr) return to_float<T>(static_cast<const T*>(p.h)[row * p.ldh + col]);
  const uint32_t z = p.h8.codes[row * p.h8.ld + col];
  const float c = p.h8.e5m2 ? unpack2<true>(z).x : unpack2<false>(z).x;
  return c * *p.h8.scale(row, col >> 7, 0);
}

// Rows too long for a block's registers: one value a lane, the rows read twice.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) ln_bwd_long_kernel(const __grid_constant__ LnBwdParams p) {
  __shared__ float2 slots[64];
  ptx::griddep_launch_dependents();
  const int32_t cols = p.cols;
  ptx::griddep_wait();
  const float inv_cols = 1.f / static_cast<float>(cols);
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const float mean = p.mean[row], rstd = p.rstd[row];
    const auto grad = [&](int32_t col) {
      const float d = to_float<T>(dy[col]);
      return p.weight != nullptr ? d * load_any(p.weight, col, p.w_dtype) : d;
    };
    float a = 0.f, b = 0.f;
#pragma unroll 4
    for (int32_t col = threadIdx.x; col < cols; col += kMaxThreads) {
      const float g = grad(col);
      a += g;
      b = fmaf(g, (h_at<T>(p, row, col) - mean) * rstd, b);
    }
    const float2 sums = row_sum2(a, b, kMaxThreads, slots, flip, 0);
    flip ^= 1;
    const float ka = sums.x * inv_cols, kb = sums.y * inv_cols;
#pragma unroll 4
    for (int32_t col = threadIdx.x; col < cols; col += kMaxThreads) {
      const float n = (h_at<T>(p, row, col) - mean) * rstd;
      const float e = p.dh != nullptr ? to_float<T>(static_cast<const T*>(p.dh)[row * p.lddh + col]) : 0.f;
      static_cast<T*>(p.dx)[row * p.lddx + col] = from_float<T>(fmaf(rstd, fmaf(-n, kb, grad(col) - ka), e));
    }
  }
}

// Partial dw and db of rows blockIdx.y, + gridDim.y, ... for 256 columns.
template <typename T>
__global__ void ln_bwd_long_dw_kernel(const __grid_constant__ LnBwdParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int32_t col = blockIdx.x * blockDim.x + threadIdx.x;
  if (col >= p.cols) return;
  float w = 0.f, b = 0.f;
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const float d = to_float<T>(static_cast<const T*>(p.dy)[row * p.lddy + col]);
    w = fmaf(d, (h_at<T>(p, row, col) - p.mean[row]) * p.rstd[row], w);
    b += d;
  }
  p.partials[static_cast<int64_t>(blockIdx.y) * 2 * p.cols + col] = w;
  p.partials[(static_cast<int64_t>(blockIdx.y) * 2 + 1) * p.cols + col] = b;
}

template <typename T, int C, int R, bool H8>
cudaError_t launch_ln_bwd_r(const LnBwdParams& p, const RowShape& s, int blocks, cudaStream_t st) {
  constexpr size_t smem = static_cast<size_t>(bwd_depth<T, C, R>()) * (kRowThreads / 32) * C * 3 * WarpRow<T>::kBytes;
  // (the row groups' sums take the ring's place)
  static_assert(smem >= kRowThreads * C * 8 * 4 + 16 * 32, "the ring holds a block's sums");
  const cudaError_t e = allow_smem<ln_bwd_kernel<T, C, R, H8>>();
  if (e != cudaSuccess) return e;
  return launch_pdl(ln_bwd_kernel<T, C, R, H8>, dim3(blocks), dim3(s.per * s.tpr), smem, st, p, s.tpr);
}

template <typename T, int C>
cudaError_t launch_ln_bwd_c(const LnBwdParams& p, int lie, const RowShape& s, int blocks, cudaStream_t st) {
  if (p.h8.codes != nullptr)
    return lie == ROWS_ALIGNED ? launch_ln_bwd_r<T, C, ROWS_ALIGNED, true>(p, s, blocks, st)
                               : launch_ln_bwd_r<T, C, ROWS_ANY, true>(p, s, blocks, st);
  if (lie == ROWS_ALIGNED) return launch_ln_bwd_r<T, C, ROWS_ALIGNED, false>(p, s, blocks, st);
  if (lie == ROWS_ALIKE) return launch_ln_bwd_r<T, C, ROWS_ALIKE, false>(p, s, blocks, st);
  return launch_ln_bwd_r<T, C, ROWS_ANY, false>(p, s, blocks, st);
}

template <typename T>
cudaError_t launch_ln_bwd_t(const LnBwdParams& p, int sms, cudaStream_t st) {
  int blocks = ln_bwd_blocks(p.rows, sms);
  cudaError_t e;
  if (p.rows == 0) {
    // no rows: dw and db are zero
  } else if (p.cols <= kMaxCols) {
    int lie = p.rows_lie;
    int64_t chunks = (p.cols + 7) / 8;
    if (lie == ROWS_ALIKE) {
      const int64_t more = alike_chunks(p.cols, sizeof(T));
      if (more * 8 <= kMaxCols && sms >= 8) chunks = more;
      else lie = ROWS_ANY;
    }
    // two chunks a thread up to the block's threads, four beyond (see launch_norm_bwd_t)
    const bool four = sizeof(T) == 2 && (lie == ROWS_ALIKE || whole_warps(chunks, 4) * 3 <= kRowThreads);
    const RowShape s = many_registers(chunks, four ? kRowThreads : 2 * kRowThreads, p.rows, sms < 64 ? sms : 64);
    const int64_t want = (p.rows + s.per - 1) / s.per;
    if (want < blocks) blocks = static_cast<int>(want);
    if (lie == ROWS_ALIKE) blocks = alike_blocks(p.rows, s.per, blocks);
    e = s.c == 1   ? launch_ln_bwd_c<T, 1>(p, lie, s, blocks, st)
        : s.c == 2 ? launch_ln_bwd_c<T, 2>(p, lie, s, blocks, st)
                   : launch_ln_bwd_c<T, 4>(p, lie, s, blocks, st);
    if (e != cudaSuccess) return e;
  } else {
    // dw and db first: dx may overwrite dy or h
    if (p.partials != nullptr) {
      e = launch_pdl(ln_bwd_long_dw_kernel<T>, dim3((p.cols + 255) / 256, blocks), dim3(256), 0, st, p);
      if (e != cudaSuccess) return e;
    }
    e = launch_pdl(ln_bwd_long_kernel<T>, dim3(static_cast<unsigned>(p.rows < 65536 ? p.rows : 65536)),
                   dim3(kMaxThreads), 0, st, p);
    if (e != cudaSuccess) return e;
  }
  return p.partials == nullptr ? cudaSuccess : launch_ln_bwd_sum(p, blocks, st);
}

#define GGE_LN_INSTANTIATE(T)                                             \
  template cudaError_t launch_ln_f<T>(const LnParams&, int, cudaStream_t); \
  template cudaError_t launch_ln_bwd_t<T>(const LnBwdParams&, int, cudaStream_t);

}  // namespace b128
}  // namespace gge
