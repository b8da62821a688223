// RMS norm with the residual's addition, and its backward.
//
//   h = round(x + residual)            (h = x without a residual)
//   inv = 1 / sqrt(mean(h^2) + eps)    y = (h inv) w
//
// The sums run in fp32.  y is rounded once to its 16-bit type, or quantised from
// fp32 to codes and block scales.
//
// Backward, for dy and the saved h and inv (dh: the gradient that reaches h
// directly, along the residual stream):
//   g = dy w    dx = inv (g - h inv^2 mean(g h)) + dh    dw = sum over rows of dy (h inv)
//
// Both are bound by memory: a row is read once into registers, reduced, and
// written from there.
#include "../gge_ptx.cuh"
#include "lowp_launch.h"
#include "mx_format.cuh"

namespace gge {
namespace lowp {
namespace {

using namespace mx;

constexpr int kBlockThreads = 256;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the `tpr` threads (a multiple of 32) that share a row.  `slots` is
// shared memory for one float a warp; `flip` alternates between its two halves,
// so one barrier a row is enough.  Every thread of the block calls it.
__device__ __forceinline__ float row_sum(float v, int tpr, float* slots, int flip) {
  v = warp_sum(v);
  if (tpr == 32) return v;
  const int warp = threadIdx.x >> 5;
  const int per = tpr >> 5;
  float* s = slots + flip * 32;
  if ((threadIdx.x & 31) == 0) s[warp] = v;
  __syncthreads();
  const int first = warp / per * per;
  float t = 0.f;
  for (int i = 0; i < per; ++i) t += s[first + i];
  return t;
}

// ------------------------------------------------------------ forward

// A row is spread over `tpr` threads; thread i holds the 8-value chunks i, i + tpr, ...
template <typename T, int C, int FMT>
__global__ void __launch_bounds__(C == 4 ? 512 : 1024) norm_kernel(const __grid_constant__ NormParams p, int tpr) {
  __shared__ float slots[64];
  ptx::griddep_launch_dependents();
  const int per_block = blockDim.x / tpr;
  const int sub = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int32_t cols = p.cols;
  QuantOut q{p.q.codes, p.q.ld, p.q.scales, p.q.kgroups, p.q.tensor_scale, p.q.values, p.q.ldv,
             p.q.v_dtype, p.q.v_vec};
  ptx::griddep_wait();
  const float tscale = (FMT == FMT_NVFP4 && q.tensor_scale) ? *q.tensor_scale : 1.f;
  const T* x = static_cast<const T*>(p.x);
  const T* res = static_cast<const T*>(p.residual);
  int flip = 0;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * per_block; row0 < p.rows;
       row0 += static_cast<int64_t>(gridDim.x) * per_block) {
    const int64_t row = row0 + sub;
    const bool live = row < p.rows;
    float v[C][8];
    float ss = 0.f;
    Raw8<T> xr[C], rr[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int32_t col = (t + c * tpr) * 8;
      if (live && col + 8 <= cols) {
        xr[c] = load8(x + row * p.ldx + col);
        if (res != nullptr) rr[c] = load8(res + row * p.ldr + col);
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int32_t col = (t + c * tpr) * 8;
      if (live && col + 8 <= cols) {
        widen(xr[c], v[c]);
        if (res != nullptr) {
          float r[8];
          widen(rr[c], r);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[c][i] += r[i];
          const Raw8<T> h = narrow<T>(v[c]);
          widen(h, v[c]);
          if (p.h != nullptr) store8(static_cast<T*>(p.h) + row * p.ldh + col, h);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[c][i] = 0.f;
          if (live && col + i < cols) {  // the row's last, partly filled chunk
            float a = to_float<T>(x[row * p.ldx + col + i]);
            if (res != nullptr) {
              const T h = from_float<T>(a + to_float<T>(res[row * p.ldr + col + i]));
              a = to_float<T>(h);
              if (p.h != nullptr) static_cast<T*>(p.h)[row * p.ldh + col + i] = h;
            }
            v[c][i] = a;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[c][i], v[c][i], ss);
    }
    ss = row_sum(ss, tpr, slots, flip);
    flip ^= 1;
    const float inv = 1.f / sqrtf(ss / static_cast<float>(cols) + p.eps);
    if (live && t == 0 && p.inv != nullptr) p.inv[row] = inv;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int32_t col = (t + c * tpr) * 8;
      float w[8];
      if (col + 8 <= cols) {
        load8_any(p.weight, col, p.w_dtype, w);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = col + i < cols ? load_any(p.weight, col + i, p.w_dtype) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = (v[c][i] * inv) * w[i];
      if (p.y != nullptr && live) {
        T* y = static_cast<T*>(p.y) + row * p.ldy + col;
        if (col + 8 <= cols) {
          store8(y, narrow<T>(v[c]));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (col + i < cols) y[i] = from_float<T>(v[c][i]);
        }
      }
      if constexpr (FMT != FMT_NONE)
        quantise_chunk<FMT>(q, v[c], row, col, cols, tscale,
                            live && col < q.kgroups * Fmt<FMT>::kGroup);
    }
  }
}

// Any alignment and any length: one value a lane, so that loads of rows that
// start anywhere still fill whole sectors; the second pass reads the row again
// (from L1).  A block is a warp's 32 (or half a warp's 16) lanes.
template <typename T, int FMT>
__global__ void norm_any_kernel(const __grid_constant__ NormParams p, int tpr) {
  __shared__ float slots[64];
  ptx::griddep_launch_dependents();
  const int per_block = blockDim.x / tpr;
  const int sub = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int lane = threadIdx.x & 31;
  const int32_t cols = p.cols;
  ptx::griddep_wait();
  const float tscale = (FMT == FMT_NVFP4 && p.q.tensor_scale) ? *p.q.tensor_scale : 1.f;
  const T* x = static_cast<const T*>(p.x);
  const T* res = static_cast<const T*>(p.residual);
  int flip = 0;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * per_block; row0 < p.rows;
       row0 += static_cast<int64_t>(gridDim.x) * per_block) {
    const int64_t row = row0 + sub;
    const bool live = row < p.rows;
    float ss = 0.f;
    auto value = [&](int32_t col, bool write) {
      float a = to_float<T>(x[row * p.ldx + col]);
      if (res != nullptr) {
        const T h = from_float<T>(a + to_float<T>(res[row * p.ldr + col]));
        if (write && p.h != nullptr) static_cast<T*>(p.h)[row * p.ldh + col] = h;
        a = to_float<T>(h);
      }
      return a;
    };
    if (live) {
#pragma unroll 4
      for (int32_t col = t; col < cols; col += tpr) {
        const float a = value(col, false);
        ss = fmaf(a, a, ss);
      }
    }
    ss = row_sum(ss, tpr, slots, flip);
    flip ^= 1;
    const float inv = 1.f / sqrtf(ss / static_cast<float>(cols) + p.eps);
    if (live && t == 0 && p.inv != nullptr) p.inv[row] = inv;
    // columns up to the end of the last scale word (whole warps take part)
    const int32_t end = FMT == FMT_NONE ? cols : static_cast<int32_t>(p.q.kgroups) * 128;
    for (int32_t col = t; col - lane < end; col += tpr) {
      float a = 0.f;
      if (live && col < cols) {
        a = (value(col, true) * inv) * load_any(p.weight, col, p.w_dtype);
        if (p.y != nullptr) static_cast<T*>(p.y)[row * p.ldy + col] = from_float<T>(a);
      }
      if constexpr (FMT != FMT_NONE) {
        constexpr int kLanes = Fmt<FMT>::kBlock;
        uint32_t amax = abs_bits(a);
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float factor;
        uint32_t s = block_scale<FMT>(amax, tscale, factor);
        const float unit = scale_value<FMT>(s);
        const int32_t block = col / Fmt<FMT>::kBlock;
        const float c = scaled(a, factor);
        float back;
        if constexpr (FMT == FMT_MXFP8) {
          const uint32_t code = pack_e4m3x4(c, 0.f, 0.f, 0.f) & 0xffu;
          if (live && col < ((cols + 31) & ~31)) p.q.codes[row * p.q.ld + col] = static_cast<uint8_t>(code);
          back = e4m3x2_to_float2(code).x;
        } else {
          const float next = __shfl_down_sync(0xffffffffu, c, 1);
          const float two[8] = {c, next, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          const uint32_t code = pack_e2m1x8(two) & 0xffu;
          if (live && (lane & 1) == 0 && col < ((cols + 31) & ~31))
            p.q.codes[row * p.q.ld + (col >> 1)] = static_cast<uint8_t>(code);
          back = e2m1x2_to_float2(code).x;
        }
        if (live && lane % kLanes == 0 && block < p.q.kgroups * 4)
          p.q.scales[scale_word(row, block >> 2, p.q.kgroups) + (block & 3)] =
              static_cast<uint8_t>(col < cols ? s : 0u);
        if (live && p.q.values != nullptr && col < cols) {
          back *= unit;
          if constexpr (FMT == FMT_NVFP4) back *= tscale;
          store_any(p.q.values, row * p.q.ldv + col, p.q.v_dtype, back);
        }
      }
    }
  }
}

// Threads a row and chunks a thread for a row of `chunks` 8-value chunks.
struct RowShape {
  int tpr, c;
};
RowShape row_shape(int64_t chunks, int64_t rows, int sms) {
  // few rows: more threads a row (latency); many: four chunks a thread, so that
  // each thread has several loads in flight and rows a block reduce cheaply
  const int most = rows <= 2 * sms ? 1 : 4;
  RowShape s{32, 1};
  while (s.tpr < (most == 4 ? 512 : 1024) && static_cast<int64_t>(s.tpr) * most < chunks) s.tpr *= 2;
  while (static_cast<int64_t>(s.tpr) * s.c < chunks) s.c *= 2;  // at most 1024 x 2 or 512 x 4
  return s;
}

template <typename T, int FMT>
cudaError_t launch_norm_t(const NormParams& p, int sms, cudaStream_t st) {
  const int64_t group = FMT == FMT_NONE ? 8 : Fmt<FMT == FMT_NONE ? 0 : FMT>::kGroup;
  const int64_t chunks = (p.cols + group - 1) / group * group / 8;
  if (p.vec && chunks <= 2 * 1024) {
    const RowShape s = row_shape(chunks, p.rows, sms);
    const int block = s.tpr > kBlockThreads ? s.tpr : kBlockThreads;
    const int per = block / s.tpr;
    const int64_t want = (p.rows + per - 1) / per;
    const int grid = static_cast<int>(want < static_cast<int64_t>(sms) * 64 ? want : static_cast<int64_t>(sms) * 64);
    if (s.c == 1) return launch_pdl(norm_kernel<T, 1, FMT>, dim3(grid), dim3(block), 0, st, p, s.tpr);
    if (s.c == 2) return launch_pdl(norm_kernel<T, 2, FMT>, dim3(grid), dim3(block), 0, st, p, s.tpr);
    return launch_pdl(norm_kernel<T, 4, FMT>, dim3(grid), dim3(block), 0, st, p, s.tpr);
  }
  int tpr = 32;
  while (tpr < 1024 && tpr * 16 < p.cols) tpr *= 2;
  const int block = tpr > kBlockThreads ? tpr : kBlockThreads;
  const int per = block / tpr;
  const int64_t want = (p.rows + per - 1) / per;
  const int grid = static_cast<int>(want < static_cast<int64_t>(sms) * 64 ? want : static_cast<int64_t>(sms) * 64);
  return launch_pdl(norm_any_kernel<T, FMT>, dim3(grid), dim3(block), 0, st, p, tpr);
}

template <typename T>
cudaError_t launch_norm_f(const NormParams& p, int sms, cudaStream_t st) {
  switch (p.q.format) {
    case FMT_MXFP8: return launch_norm_t<T, FMT_MXFP8>(p, sms, st);
    case FMT_MXFP4: return launch_norm_t<T, FMT_MXFP4>(p, sms, st);
    case FMT_NVFP4: return launch_norm_t<T, FMT_NVFP4>(p, sms, st);
    default: return launch_norm_t<T, FMT_NONE>(p, sms, st);
  }
}

// ----------------------------------------------------------- backward

// Each block walks rows blockIdx.x, + gridDim.x, ... and keeps its share of dw
// in registers; at its end it leaves them as one row of partial sums.
template <typename T, int C>
__global__ void __launch_bounds__(1024) norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
  __shared__ float slots[64];
  ptx::griddep_launch_dependents();
  const int t = threadIdx.x, tpr = blockDim.x;
  const int32_t cols = p.cols;
  ptx::griddep_wait();
  float dw[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0.f;
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const T* h = static_cast<const T*>(p.h) + row * p.ldh;
    Raw8<T> dyr[C], hr[C], er[C];
    const float inv = p.inv[row];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int32_t col = (t + c * tpr) * 8;
      if (col < cols) {
        dyr[c] = load8(dy + col);
        hr[c] = load8(h + col);
        if (p.dh != nullptr) er[c] = load8(static_cast<const T*>(p.dh) + row * p.lddh + col);
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int32_t col = (t + c * tpr) * 8;
      if (col < cols) {
        float a[8], b[8], w[8];
        widen(dyr[c], a);
        widen(hr[c], b);
        load8_any(p.weight, col, p.w_dtype, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw[c][i] = fmaf(a[i], b[i] * inv, dw[c][i]);
          dot = fmaf(a[i] * w[i], b[i], dot);
        }
      }
    }
    dot = row_sum(dot, tpr, slots, flip);
    flip ^= 1;
    const float k = dot / static_cast<float>(cols) * inv * inv;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int32_t col = (t + c * tpr) * 8;
      if (col < cols) {
        float a[8], b[8], w[8], e[8];
        widen(dyr[c], a);
        widen(hr[c], b);
        load8_any(p.weight, col, p.w_dtype, w);
        if (p.dh != nullptr) {
          widen(er[c], e);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = fmaf(inv, fmaf(-b[i], k, a[i] * w[i]), e[i]);
        store8(static_cast<T*>(p.dx) + row * p.lddx + col, narrow<T>(a));
      }
    }
  }
  if (p.dw != nullptr) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int32_t col = (t + c * tpr) * 8;
      if (col < cols) store8_any(p.partials, static_cast<int64_t>(blockIdx.x) * cols + col, 4, dw[c]);
    }
  }
}

// Any alignment and any length: one value a lane, the rows read twice.  dw is
// summed by columns in a kernel of its own (norm_bwd_dw_any_kernel).
template <typename T>
__global__ void norm_bwd_any_kernel(const __grid_constant__ NormBwdParams p) {
  __shared__ float slots[64];
  ptx::griddep_launch_dependents();
  const int t = threadIdx.x, tpr = blockDim.x;
  const int32_t cols = p.cols;
  ptx::griddep_wait();
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const T* h = static_cast<const T*>(p.h) + row * p.ldh;
    const float inv = p.inv[row];
    float dot = 0.f;
#pragma unroll 4
    for (int32_t col = t; col < cols; col += tpr)
      dot = fmaf(to_float<T>(dy[col]) * load_any(p.weight, col, p.w_dtype), to_float<T>(h[col]), dot);
    dot = row_sum(dot, tpr, slots, flip);
    flip ^= 1;
    const float k = dot / static_cast<float>(cols) * inv * inv;
#pragma unroll 4
    for (int32_t col = t; col < cols; col += tpr) {
      const float g = to_float<T>(dy[col]) * load_any(p.weight, col, p.w_dtype);
      const float e = p.dh != nullptr ? to_float<T>(static_cast<const T*>(p.dh)[row * p.lddh + col]) : 0.f;
      static_cast<T*>(p.dx)[row * p.lddx + col] =
          from_float<T>(fmaf(inv, fmaf(-to_float<T>(h[col]), k, g), e));
    }
  }
}

// Partial dw of rows blockIdx.y, + gridDim.y, ... for 256 columns.
template <typename T>
__global__ void norm_bwd_dw_any_kernel(const __grid_constant__ NormBwdParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int32_t col = blockIdx.x * blockDim.x + threadIdx.x;
  if (col >= p.cols) return;
  float s = 0.f;
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y)
    s = fmaf(to_float<T>(static_cast<const T*>(p.dy)[row * p.lddy + col]),
             to_float<T>(static_cast<const T*>(p.h)[row * p.ldh + col]) * p.inv[row], s);
  p.partials[static_cast<int64_t>(blockIdx.y) * p.cols + col] = s;
}

// dw[col] = the partial rows' sum: 32 columns a block, eight warps a column
// share the rows, joined in a fixed order.
__global__ void norm_bwd_dw_kernel(const float* partials, int blocks, int32_t cols, float* dw) {
  __shared__ float part[8][33];
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t col = blockIdx.x * 32 + lane;
  ptx::griddep_wait();
  float s = 0.f;
  if (col < cols) {
#pragma unroll 4
    for (int b = warp; b < blocks; b += 8) s += partials[static_cast<int64_t>(b) * cols + col];
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < cols) {
    float v = part[0][lane];
#pragma unroll
    for (int i = 1; i < 8; ++i) v += part[i][lane];
    dw[col] = v;
  }
}

template <typename T>
cudaError_t launch_norm_bwd_t(const NormBwdParams& p, int sms, cudaStream_t st) {
  const int blocks = norm_bwd_blocks(p.rows, sms);
  const int64_t chunks = (p.cols + 7) / 8;
  cudaError_t e;
  if (p.rows == 0) {
    // no rows: dw is zero
  } else if (p.vec && p.cols % 8 == 0 && chunks <= 2 * 1024) {
    int c = 1, threads = 32;
    while (threads < 1024 && static_cast<int64_t>(threads) * 2 < chunks) threads *= 2;
    while (static_cast<int64_t>(threads) * c < chunks) c *= 2;
    if (c == 1) e = launch_pdl(norm_bwd_kernel<T, 1>, dim3(blocks), dim3(threads), 0, st, p);
    else e = launch_pdl(norm_bwd_kernel<T, 2>, dim3(blocks), dim3(threads), 0, st, p);
    if (e != cudaSuccess) return e;
  } else {
    int threads = 32;
    while (threads < 1024 && threads * 8 < p.cols) threads *= 2;
    // dw first: dx may overwrite dy or h
    if (p.dw != nullptr) {
      e = launch_pdl(norm_bwd_dw_any_kernel<T>, dim3((p.cols + 255) / 256, blocks), dim3(256), 0, st, p);
      if (e != cudaSuccess) return e;
    }
    e = launch_pdl(norm_bwd_any_kernel<T>, dim3(static_cast<unsigned>(p.rows < 65536 ? p.rows : 65536)),
                   dim3(threads), 0, st, p);
    if (e != cudaSuccess) return e;
  }
  if (p.dw == nullptr) return cudaSuccess;
  return launch_pdl(norm_bwd_dw_kernel, dim3((p.cols + 31) / 32), dim3(256), 0, st,
                    static_cast<const float*>(p.partials), blocks, p.cols, p.dw);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, int sms, cudaStream_t st) {
  if (p.dtype == 0) return launch_norm_f<__nv_bfloat16>(p, sms, st);
  if (p.dtype == 1) return launch_norm_f<__half>(p, sms, st);
  return launch_norm_f<float>(p, sms, st);
}

int norm_bwd_blocks(int64_t rows, int sms) {
  const int64_t most = 2 * static_cast<int64_t>(sms);
  return static_cast<int>(rows < most ? rows : most);
}

cudaError_t launch_norm_bwd(const NormBwdParams& p, int sms, cudaStream_t st) {
  if (p.dtype == 0) return launch_norm_bwd_t<__nv_bfloat16>(p, sms, st);
  if (p.dtype == 1) return launch_norm_bwd_t<__half>(p, sms, st);
  return launch_norm_bwd_t<float>(p, sms, st);
}

}  // namespace lowp
}  // namespace gge
