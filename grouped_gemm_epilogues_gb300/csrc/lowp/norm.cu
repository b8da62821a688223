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
// Both are bound by memory.  Blocks walk the rows with a grid stride; cp.async
// keeps the next rows on their way to shared memory while a row is reduced in
// registers and written, so every value is read once.  What limits them beside the
// DRAM is instruction issue, hence the packed fp32 operations and, where the rows' place
// in memory allows it, forms without the shifting of rows.cuh (Rows).  Measured: bf16
// 16384 x 8192 with residual, mxfp8 and its values 190 us (6.4 TB/s, 95 % of a copy's
// rate; the first version, without copies ahead and packed arithmetic, 273).  Rows that
// start on any 2 bytes, fp16 16000 x 1999: 26 us alike (4.9 TB/s), 40 shifted.  Backward 16384
// x 4096 with dh 85 us (6.3 TB/s, 94 %), bf16 24000 x 1999 70 us (5.5 TB/s).  Codes
// without their values: mxfp8 16384 x 8192 159 us (5.9 TB/s, 89 %).
#include <numeric>

#include "lowp_launch.h"
#include "rows.cuh"

namespace gge {
namespace lowp {
namespace {

using namespace mx;

constexpr int kMaxThreads = 1024;
// Where the weights (and dw) stay in registers with the row, over its sum, a block has
// half the threads with twice the registers, and up to four chunks of 8 values each.
constexpr int kRowThreads = 512;

// Rows of `bytes` in an SM's shared memory: the one at work and those on their way.
// (A depth known at run time only, up to eight rows: 10 % slower for 8000 x 4096.)
constexpr int ring_depth(int bytes, int most) {
  return 210 * 1024 / bytes < most ? 210 * 1024 / bytes : most;
}
constexpr int kMaxCols = kMaxThreads * 2 * 8;  // longer rows take the *_long kernels

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the `tpr` threads (a multiple of 32) that share a row, the block's
// `sub`-th.  `slots` is shared memory for one float a warp, twice; `flip`
// alternates between the two, so one barrier a row is enough.
__device__ __forceinline__ float row_sum(float v, int tpr, float* slots, int flip, int sub) {
  v = warp_sum(v);
  if (tpr == 32) return v;
  const int warp = threadIdx.x >> 5;
  const int per = tpr >> 5;
  float* s = slots + flip * 32;
  if ((threadIdx.x & 31) == 0) s[warp] = v;
  // (a barrier of its own for each row group: the groups do not run in step, and
  // barrier 0 is the whole block's)
  asm volatile("bar.sync %0, %1;" ::"r"(sub + 1), "r"(tpr) : "memory");
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < per ? s[sub * per + lane] : 0.f);
}

// Eight weights from column col on (zeros outside the row).
__device__ __forceinline__ void load_weight(const void* w, int32_t dtype, int32_t vec, int32_t col,
                                            int32_t cols, float2 (&v)[4]) {
  if (vec && col + 8 <= cols) {
    if (dtype == 0) widen(load8(static_cast<const __nv_bfloat16*>(w) + col), v);
    else if (dtype == 1) widen(load8(static_cast<const __half*>(w) + col), v);
    else widen(load8(static_cast<const float*>(w) + col), v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int32_t a = col + 2 * i, b = a + 1;
      v[i].x = a >= 0 && a < cols ? load_any(w, a, dtype) : 0.f;
      v[i].y = b >= 0 && b < cols ? load_any(w, b, dtype) : 0.f;
    }
  }
}

// A lane's 8 values, those past the row's end set to zero.
template <typename T>
__device__ __forceinline__ void clear_past(Raw8<T>& r, int32_t col, int32_t cols) {
  if (col + 8 <= cols) return;
  T* t = reinterpret_cast<T*>(&r);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col + i >= cols) t[i] = from_float<T>(0.f);
}

template <typename T>
__device__ __forceinline__ int32_t row_skew(const void* row) {
  return static_cast<int32_t>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}

// The first k (0 to 7) set to zero.
template <typename T>
__device__ __forceinline__ void clear_front(Raw8<T>& r, int32_t k) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
  for (int j = 0; j < 2 * static_cast<int>(sizeof(T)); ++j) {
    const int32_t bits = 8 * static_cast<int>(sizeof(T)) * k - 32 * j;  // of word j
    w[j] &= __funnelshift_lc(0u, 0xffffffffu, static_cast<uint32_t>(max(bits, 0)));
  }
}

// One tensor's rows on their way through shared memory, for one warp: in ANY the
// warp does it together, otherwise a lane copies and reads its own pieces only.
template <typename T, int R>
struct RowReader {
  const T* next;  // this lane's chunk 0 of the next row to copy

  __device__ __forceinline__ void init(const void* base, int64_t ld, int64_t row, int32_t col) {
    next = static_cast<const T*>(base) + row * ld + col;
  }
  // Once a buffer (not ANY): a lane's pieces past the row's end stay zero.
  static __device__ __forceinline__ void clear(uint32_t dst, int32_t col, int32_t cols) {
    constexpr int P = WarpRow<T>::kPieces;
    if constexpr (R != ROWS_ANY) {
#pragma unroll
      for (int j = 0; j < P; ++j)
        if (col + j * static_cast<int32_t>(16 / sizeof(T)) >= cols)
          ptx::st_shared_v4(dst + 16u * ((threadIdx.x & 31) * P + j), make_uint4(0u, 0u, 0u, 0u));
    }
  }
  // Copy chunk c (`over` columns after chunk 0) of that row to this warp's `dst`.
  // `first`: nothing may be read in front of the row.
  __device__ __forceinline__ void copy(uint32_t dst, int32_t col, int32_t c, int32_t over, int32_t cols,
                                       bool first) const {
    constexpr int P = WarpRow<T>::kPieces;
    const int lane = threadIdx.x & 31;
    const int32_t left = (cols - col) * static_cast<int32_t>(sizeof(T));
    if constexpr (R != ROWS_ANY) {
      if (R == ROWS_ALIKE && c == 0 && first && col < 0) {  // (one thread of the launch's first rows)
        const T* at = next + over;
        for (int32_t i = -col; i < min(static_cast<int32_t>(16 / sizeof(T)), cols - col); ++i) {
          if constexpr (sizeof(T) == 2)
            ptx::st_shared_u16(dst + 16u * (lane * P) + 2 * i, *reinterpret_cast<const uint16_t*>(at + i));
          else
            ptx::st_shared_u32(dst + 16u * (lane * P) + 4 * i, *reinterpret_cast<const uint32_t*>(at + i));
        }
      }
#pragma unroll
      for (int j = 0; j < P; ++j) {
        if (R == ROWS_ALIKE && c == 0 && j == 0 && first && col < 0) continue;
        // (bytes past the row's end are zero-filled; none are read)
        if (left > 16 * j)
          ptx::cp_async_16(dst + 16u * (lane * P + j), next + over + j * (16 / sizeof(T)),
                           static_cast<uint32_t>(min(16, left - 16 * j)));
      }
    } else {
      copy_row(dst, next + over, left, first && col == lane * 8);
    }
  }
};

// A lane's 8 values of the copied chunk c of the row that starts at `row`; zeros where the
// chunk leaves the row.
template <typename T, int R>
__device__ __forceinline__ Raw8<T> take_chunk(uint32_t src, int32_t c, const T* row, int32_t col, int32_t cols) {
  constexpr int P = WarpRow<T>::kPieces;
  if constexpr (R != ROWS_ANY) {
    Raw8<T> r;
#pragma unroll
    for (int j = 0; j < P; ++j) r.w[j] = ptx::ld_shared_v4(src + 16u * ((threadIdx.x & 31) * P + j));
    if (R == ROWS_ALIKE && c == 0 && col < 0) {
      clear_front(r, -col);
      clear_past(r, col, cols);
    }
    return r;
  } else {
    Raw8<T> r = take_row<T>(src, static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row)) & 15u);
    clear_past(r, col, cols);
    return r;
  }
}

template <typename T, int R>
__device__ __forceinline__ void put_chunk(T* row, int32_t c, int32_t col, int32_t cols, const Raw8<T>& v) {
  if (R == ROWS_ALIKE && c == 0 && col < 0) {
    if (col + 8 <= cols) {
      store_from(row + col, -col, v);
    } else {  // (a row shorter than 8)
      const T* t = reinterpret_cast<const T*>(&v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= -col && col + i < cols) row[col + i] = t[i];
    }
  } else if constexpr (R != ROWS_ANY) {
    store_row8_aligned(row, col, cols, v);
  } else {
    store_row8(row, col, cols, v);
  }
}

// A launch's blocks such that a row group's rows are a multiple of 8 apart (of which
// every skew has an equal), if it takes more than one; 0 if there are too few.
int alike_blocks(int64_t rows, int per_block, int64_t blocks) {
  if (rows <= blocks * per_block) return static_cast<int>(blocks);
  const int unit = 8 / std::gcd(8, per_block);
  return static_cast<int>(blocks / unit * unit);
}

// ------------------------------------------------------------ forward

// Threads a block has at most.  ALIKE's weights stay in registers.  The others take
// them from L1 again for each row: with codes, more warps are worth more (mxfp8 16384 x
// 8192 with residual 190 us, with 512 threads and the weights in registers 258; ALIKE,
// bf16 24000 x 1999 with residual, 83 and 64).
template <int R>
constexpr int norm_threads() {
  return R == ROWS_ALIKE ? kRowThreads : kMaxThreads;
}

// Rows in shared memory: in ALIKE, which has half the rows at work, up to four.
template <typename T, int C, int R>
constexpr int norm_depth() {
  return ring_depth(norm_threads<R>() / 32 * C * 2 * WarpRow<T>::kBytes, R == ROWS_ALIKE ? 4 : 2);
}

// A row is spread over `tpr` threads; thread i holds the 8-value chunks i, i + tpr, ...
// The block's row groups run on their own: what they share is shared memory's size.
template <typename T, int C, int FMT, int R>
__global__ void __launch_bounds__(norm_threads<R>())
    norm_kernel(const __grid_constant__ NormParams p, int tpr) {
  __shared__ float slots[64];
  extern __shared__ uint8_t ring_raw[];
  ptx::griddep_launch_dependents();
  const int per_block = blockDim.x / tpr;
  const int sub = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int32_t cols = p.cols;
  constexpr int D = norm_depth<T, C, R>();
  const bool has_res = p.residual != nullptr;
  // this warp's buffers: [row in flight][chunk][x, residual]
  constexpr uint32_t kBuf = WarpRow<T>::kBytes;
  constexpr uint32_t kRow = 2 * C * kBuf;
  const uint32_t ring = ptx::smem_addr(ring_raw) + (threadIdx.x >> 5) * kRow;
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
  ptx::griddep_wait();
  const float tscale = (FMT == FMT_NVFP4 && p.q.tensor_scale) ? *p.q.tensor_scale : 1.f;
#pragma unroll
  for (int s = 0; s < D * C * 2; ++s)
    RowReader<T, R>::clear(ring + s / (C * 2) * ring_row + s % (C * 2) * kBuf, col0 + s % (C * 2) / 2 * tpr * 8, cols);
  float2 wk[C][4];  // ALIKE: the weights stay in registers
  if constexpr (R == ROWS_ALIKE) {
#pragma unroll
    for (int c = 0; c < C; ++c) load_weight(p.weight, p.w_dtype, 0, col0 + c * tpr * 8, cols, wk[c]);
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
  for (; row < rows; row += step) {
    if constexpr (R == ROWS_ANY) __syncwarp();  // (the slot was read in the iteration before)
    start((slot + D - 1) % D);
    cp_async_wait<D - 1>();
    if constexpr (R == ROWS_ANY) __syncwarp();
    Raw8<T> h[C];
    float2 ss = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int32_t col = col0 + c * tpr * 8;
      const uint32_t src = ring + slot * ring_row + c * 2 * kBuf;
      h[c] = take_chunk<T, R>(src, c, static_cast<const T*>(p.x) + row * p.ldx, col, cols);
      if (has_res) {
        h[c] = add8(h[c], take_chunk<T, R>(src + kBuf, c, static_cast<const T*>(p.residual) + row * p.ldr, col, cols));
        if (p.h != nullptr && warp_col + c * tpr * 8 < cols)
          put_chunk<T, R>(static_cast<T*>(p.h) + row * p.ldh, c, col, cols, h[c]);
      }
      float2 v[4];
      widen(h[c], v);
#pragma unroll
      for (int i = 0; i < 4; ++i) ss = __ffma2_rn(v[i], v[i], ss);
    }
    slot = (slot + 1) % D;
    const float sum = row_sum(ss.x + ss.y, tpr, slots, flip, sub);
    flip ^= 1;
    // (rounded correctly: an error of inv moves every value of the row the same way)
    const float inv = __frsqrt_rn(fmaf(sum, inv_cols, p.eps));
    if (t == 0 && p.inv != nullptr) p.inv[row] = inv;
    uint8_t *codes = nullptr, *scales = nullptr;
    if constexpr (FMT != FMT_NONE) {
      codes = p.q.codes + row * p.q.ld;
      scales = p.q.scales + scale_word(row, 0, p.q.kgroups);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int32_t col = col0 + c * tpr * 8;
      if (c > 0 && warp_col + c * tpr * 8 >= cols) continue;
      float2 v[4], w[4];
      widen(h[c], v);
      if constexpr (R != ROWS_ALIKE) load_weight(p.weight, p.w_dtype, p.w_vec, col, cols, w);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = __fmul2_rn(__fmul2_rn(v[i], make_float2(inv, inv)), R == ROWS_ALIKE ? wk[c][i] : w[i]);
      if (p.y != nullptr) put_chunk<T, R>(static_cast<T*>(p.y) + row * p.ldy, c, col, cols, narrow<T>(v));
      if constexpr (FMT != FMT_NONE) {
        constexpr int B = Fmt<FMT>::kBlock;
        const Quantised z = quantise8<FMT>(v, tscale, col >= (cols + B - 1) / B * B);
        if (holds_word<FMT>() && col < p.q.kgroups * Fmt<FMT>::kGroup)
          *reinterpret_cast<uint32_t*>(scales + static_cast<int64_t>(col / Fmt<FMT>::kGroup) * 512) = z.word;
        if (col < ((cols + 31) & ~31)) store_codes<FMT>(codes + static_cast<int64_t>(col) * Fmt<FMT>::kBits / 8, z.codes);
        if (p.q.values != nullptr) {
          code_values<FMT>(z.codes, z.unit, tscale, v);
          store_row8_any<R == ROWS_ALIGNED>(p.q.values, row * p.q.ldv, p.q.v_dtype, col, cols, v);
        }
      }
    }
  }
}

// Rows too long for a block's registers: one value a lane, and a second pass that
// reads the row again.  A scale's block is a warp's 32 (or half a warp's 16) lanes.
// The simple form, bound by its loads of 2 bytes: bf16 8192 x 18432 with residual 662 us
// (1.8 TB/s of what it cannot do without), mxfp8 962, nvfp4 1022.
template <typename T, int FMT>
__global__ void __launch_bounds__(kMaxThreads) norm_long_kernel(const __grid_constant__ NormParams p) {
  __shared__ float slots[64];
  ptx::griddep_launch_dependents();
  const int t = threadIdx.x, tpr = blockDim.x;
  const int lane = threadIdx.x & 31;
  const int32_t cols = p.cols;
  ptx::griddep_wait();
  const float tscale = (FMT == FMT_NVFP4 && p.q.tensor_scale) ? *p.q.tensor_scale : 1.f;
  const T* x = static_cast<const T*>(p.x);
  const T* res = static_cast<const T*>(p.residual);
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    float ss = 0.f;
    auto value = [&](int64_t col, bool write) {
      float a = to_float<T>(x[row * p.ldx + col]);
      if (res != nullptr) {
        const T h = from_float<T>(a + to_float<T>(res[row * p.ldr + col]));
        if (write && p.h != nullptr) static_cast<T*>(p.h)[row * p.ldh + col] = h;
        a = to_float<T>(h);
      }
      return a;
    };
#pragma unroll 4
    for (int32_t col = t; col < cols; col += tpr) {
      const float a = value(col, false);
      ss = fmaf(a, a, ss);
    }
    ss = row_sum(ss, tpr, slots, flip, 0);
    flip ^= 1;
    const float inv = __frsqrt_rn(ss / static_cast<float>(cols) + p.eps);
    if (t == 0 && p.inv != nullptr) p.inv[row] = inv;
    // columns up to the end of the last scale word (whole warps take part)
    int64_t end = cols;
    if constexpr (FMT != FMT_NONE) end = scale_span<FMT>(p.q.kgroups);
    for (int64_t col = t; col - lane < end; col += tpr) {
      float a = 0.f;
      if (col < cols) {
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
        const int64_t block = col / Fmt<FMT>::kBlock;
        const float c = a * factor;
        float back;
        if constexpr (FMT == FMT_MXFP8) {
          const uint32_t code = pack_e4m3x4(c, 0.f, 0.f, 0.f) & 0xffu;
          if (col < ((cols + 31) & ~31)) p.q.codes[row * p.q.ld + col] = static_cast<uint8_t>(code);
          back = e4m3x2_to_float2(code).x;
        } else {
          const float next = __shfl_down_sync(0xffffffffu, c, 1);
          const float two[8] = {c, next, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          const uint32_t code = pack_e2m1x8(two) & 0xffu;
          if ((lane & 1) == 0 && col < ((cols + 31) & ~31))
            p.q.codes[row * p.q.ld + (col >> 1)] = static_cast<uint8_t>(code);
          back = e2m1x2_to_float2(code).x;
        }
        if (lane % kLanes == 0 && block < p.q.kgroups * 4)
          p.q.scales[scale_word(row, block >> 2, p.q.kgroups) + (block & 3)] =
              static_cast<uint8_t>(col < cols ? s : 0u);
        if (p.q.values != nullptr && col < cols) {
          back *= unit;
          if constexpr (FMT == FMT_NVFP4) back *= tscale;
          store_any(p.q.values, row * p.q.ldv + col, p.q.v_dtype, back);
        }
      }
    }
  }
}

// How a row is spread: chunks a thread, threads a row (whole warps), rows a block, and
// blocks an SM.  Row groups of several warps have a barrier each, of the 15 beside the
// block's.
struct RowShape {
  int c, tpr, per, blocks;
};
int whole_warps(int64_t chunks, int c) { return static_cast<int>((chunks + 32 * c - 1) / (32 * c) * 32); }

// ... with up to 64 registers a thread: blocks such that as many rows as possible are at
// work.  An SM has four quarters of 8 such warps, and a block's warps go round them.
// (1536 columns, 96 threads a row: 5 rows a block, twice, 34 us for 48 M values; 2 rows
// a block, which leaves room for four blocks, 46.)  Few rows have one chunk a thread
// (latency); many two, so that a row's barrier costs less.
RowShape many_threads(int64_t chunks, bool few) {
  RowShape s{chunks > (few ? kMaxThreads : 32) ? 2 : 1, 0, 0, 0};
  s.tpr = whole_warps(chunks, s.c);
  for (int per = 1; per * s.tpr <= kMaxThreads && (s.tpr == 32 || per <= 15); ++per) {
    const int warps = per * s.tpr / 32;
    const int blocks = 8 / ((warps + 3) / 4);
    const int now = per * blocks, best = s.per * s.blocks;
    // (blocks below 256 threads were slower at the same number of rows; above, alike)
    if (now > best || (now == best && s.per * s.tpr < 256)) s.per = per, s.blocks = blocks;
  }
  return s;
}

// ... with up to 128: one block.  Rows of more than `two` chunks have four a thread.  Few
// rows are spread over `spread` SMs, and with one a block, a row has as many threads as it
// can use.  The forward takes every SM (8 x 1999 4.3 to 2.3 us against blocks filled first);
// the backward 64, as each block leaves a row of dw's sums (152 x 1536 5.2 us, 6.1 with all
// 152; 8 x 1536 4.9 to 4.4).
RowShape many_registers(int64_t chunks, int64_t two, int64_t rows, int spread) {
  const bool few = rows <= spread;
  RowShape s{chunks > (few ? 2 * kRowThreads : two) ? 4 : (chunks > (few ? kRowThreads : 32) ? 2 : 1), 0, 0, 1};
  s.tpr = whole_warps(chunks, s.c);
  s.per = kRowThreads / s.tpr;
  const int64_t each = (rows + spread - 1) / spread;
  if (each < s.per) s.per = static_cast<int>(each);
  return s;
}

// Chunks of a row of `cols` values that starts at any skew.
int64_t alike_chunks(int64_t cols, int value_bytes) { return (cols + 16 / value_bytes - 1 + 7) / 8; }

template <typename T, int C, int FMT, int R>
cudaError_t launch_norm_c(const NormParams& p, const RowShape& s, int sms, cudaStream_t st) {
  const int block = s.per * s.tpr;
  const size_t smem = static_cast<size_t>(norm_depth<T, C, R>()) * (block / 32) * C * 2 * WarpRow<T>::kBytes;
  const cudaError_t e = allow_smem<norm_kernel<T, C, FMT, R>>();
  if (e != cudaSuccess) return e;
  // as many blocks as an SM holds, each with its share of the rows
  const int64_t resident = static_cast<int64_t>(sms) * s.blocks;
  const int64_t want = (p.rows + s.per - 1) / s.per;
  int blocks = static_cast<int>(want < resident ? want : resident);
  if (R == ROWS_ALIKE) blocks = alike_blocks(p.rows, s.per, blocks);
  return launch_pdl(norm_kernel<T, C, FMT, R>, dim3(blocks), dim3(block), smem, st, p, s.tpr);
}

template <typename T, int FMT>
cudaError_t launch_norm_t(const NormParams& p, int sms, cudaStream_t st) {
  int64_t span = (static_cast<int64_t>(p.cols) + 7) / 8 * 8;
  if constexpr (FMT != FMT_NONE) span = scale_span<FMT>(p.q.kgroups);
  if (span <= kMaxCols) {
    if constexpr (FMT == FMT_NONE) {
      const int64_t chunks = alike_chunks(p.cols, sizeof(T));
      if (p.rows_lie == ROWS_ALIKE && chunks * 8 <= kMaxCols && sms >= 8) {
        // (16 bits, 24000 x 1999, two and four: 49 and 35 us, with residual 69 and 66; 48000 x
        // 1003 49 and 36; fp32 12000 x 1999 38 and 38, with residual 66 and 71)
        const RowShape s = many_registers(chunks, sizeof(T) == 2 ? 64 : 2 * kRowThreads, p.rows, sms);
        return s.c == 1   ? launch_norm_c<T, 1, FMT, ROWS_ALIKE>(p, s, sms, st)
               : s.c == 2 ? launch_norm_c<T, 2, FMT, ROWS_ALIKE>(p, s, sms, st)
                          : launch_norm_c<T, 4, FMT, ROWS_ALIKE>(p, s, sms, st);
      }
    }
    const RowShape s = many_threads(span / 8, p.rows <= sms);
    if (p.rows_lie == ROWS_ALIGNED)
      return s.c == 1 ? launch_norm_c<T, 1, FMT, ROWS_ALIGNED>(p, s, sms, st)
                      : launch_norm_c<T, 2, FMT, ROWS_ALIGNED>(p, s, sms, st);
    return s.c == 1 ? launch_norm_c<T, 1, FMT, ROWS_ANY>(p, s, sms, st)
                    : launch_norm_c<T, 2, FMT, ROWS_ANY>(p, s, sms, st);
  }
  return launch_pdl(norm_long_kernel<T, FMT>,
                    dim3(static_cast<unsigned>(p.rows < 65536 ? p.rows : 65536)), dim3(kMaxThreads), 0, st, p);
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

// Rows in shared memory (bf16 8000 x 4096 with dh, three and four: 46.2 and 47.3 us;
// 24000 x 1999 80 and 70).
template <typename T, int C, int R>
constexpr int bwd_depth() {
  return ring_depth(kRowThreads / 32 * C * 3 * WarpRow<T>::kBytes, R == ROWS_ALIKE ? 4 : 3);
}

// A block takes as many rows at a time as its threads hold.  Each thread keeps its
// columns' share of dw in registers; at the end the block's row groups add theirs
// up and leave one row of partial sums.
template <typename T, int C, int R>
__global__ void __launch_bounds__(kRowThreads)
    norm_bwd_kernel(const __grid_constant__ NormBwdParams p, int tpr) {
  __shared__ float slots[64];
  extern __shared__ uint8_t ring_raw[];
  ptx::griddep_launch_dependents();
  // g and h stay in registers over the row's sum, or are made again from shared memory
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
  const int32_t skew = R == ROWS_ALIKE ? row_skew<T>(static_cast<const T*>(p.h) + row * p.ldh) : 0;
  const int32_t col0 = t * 8 - skew;         // chunk 0's first column
  const int32_t warp_col = col0 - lane * 8;  // and its warp's
  dy.init(p.dy, p.lddy, row, col0);
  h.init(p.h, p.ldh, row, col0);
  dh.init(p.dh, p.lddh, row, col0);
  ptx::griddep_wait();
  float2 dw[C][4];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[c][i] = make_float2(0.f, 0.f);
  float2 w[C][4];
#pragma unroll
  for (int c = 0; c < C; ++c)
    load_weight(p.weight, p.w_dtype, R == ROWS_ALIKE ? 0 : p.w_vec, col0 + c * tpr * 8, cols, w[c]);
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
        h.copy(dst + kBuf, col, c, over, cols, ahead * p.ldh < 8);
        if (has_dh) dh.copy(dst + 2 * kBuf, col, c, over, cols, ahead * p.lddh < 8);
      }
      dy.next += static_cast<int64_t>(step) * p.lddy;
      h.next += static_cast<int64_t>(step) * p.ldh;
      dh.next += static_cast<int64_t>(step) * p.lddh;
    }
    ahead += step;
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s + 1 < D; ++s) start(s);
  const float inv_cols = 1.f / static_cast<float>(cols);
  int slot = 0, flip = 0;
  float inv_next = row < rows ? p.inv[row] : 0.f;
  for (; row < rows; row += step) {
    if constexpr (R == ROWS_ANY) __syncwarp();
    start((slot + D - 1) % D);
    const float inv = inv_next;
    if (row + step < rows) inv_next = p.inv[row + step];
    const float2 inv2 = make_float2(inv, inv);
    cp_async_wait<D - 1>();
    if constexpr (R == ROWS_ANY) __syncwarp();
    const uint32_t src = ring + slot * ring_row;
    Raw8<T> hr[kKeep ? C : 1];
    float2 g[kKeep ? C : 1][4];
    float2 dot = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int32_t col = col0 + c * tpr * 8;
      float2 hv[4];
      float2(&z)[4] = g[kKeep ? c : 0];
      widen(take_chunk<T, R>(src + c * 3 * kBuf, c, static_cast<const T*>(p.dy) + row * p.lddy, col, cols), z);
      Raw8<T>& raw = hr[kKeep ? c : 0];
      raw = take_chunk<T, R>(src + c * 3 * kBuf + kBuf, c, static_cast<const T*>(p.h) + row * p.ldh, col, cols);
      widen(raw, hv);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dw[c][i] = __ffma2_rn(z[i], __fmul2_rn(hv[i], inv2), dw[c][i]);
        z[i] = __fmul2_rn(z[i], w[c][i]);
        dot = __ffma2_rn(z[i], hv[i], dot);
      }
    }
    const float sum = row_sum(dot.x + dot.y, tpr, slots, flip, sub);
    flip ^= 1;
    const float k = -(sum * inv_cols) * inv * inv;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int32_t col = col0 + c * tpr * 8;
      if (warp_col + c * tpr * 8 >= cols) continue;
      float2 v[4];
      float2(&z)[4] = g[kKeep ? c : 0];
      if constexpr (!kKeep) {
        hr[0] = take_chunk<T, R>(src + c * 3 * kBuf + kBuf, c, static_cast<const T*>(p.h) + row * p.ldh, col, cols);
        widen(take_chunk<T, R>(src + c * 3 * kBuf, c, static_cast<const T*>(p.dy) + row * p.lddy, col, cols), z);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = __fmul2_rn(z[i], w[c][i]);
      }
      widen(hr[kKeep ? c : 0], v);
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = __fmul2_rn(inv2, __ffma2_rn(v[i], make_float2(k, k), z[i]));
      if (has_dh) {
        widen(take_chunk<T, R>(src + c * 3 * kBuf + 2 * kBuf, c, static_cast<const T*>(p.dh) + row * p.lddh, col, cols), v);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = __fadd2_rn(z[i], v[i]);
      }
      put_chunk<T, R>(static_cast<T*>(p.dx) + row * p.lddx, c, col, cols, narrow<T>(z));
    }
    slot = (slot + 1) % D;
  }
  if (p.dw == nullptr) return;
  // the row groups' sums, added in their order
  cp_async_wait<0>();
  __syncthreads();
  float* sums = reinterpret_cast<float*>(ring_raw);  // [group][8 + column]
  const int32_t pitch = tpr * C * 8 + 8;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float* at = sums + sub * pitch + 8 + col0 + c * tpr * 8 + 2 * i;
      if constexpr (R == ROWS_ALIKE) at[0] = dw[c][i].x, at[1] = dw[c][i].y;
      else *reinterpret_cast<float2*>(at) = dw[c][i];
    }
  __syncthreads();
  for (int32_t col = threadIdx.x; col < cols; col += blockDim.x) {
    float s = 0.f;
    for (int g = 0; g < per_block; ++g) s += sums[g * pitch + 8 + col];
    p.partials[static_cast<int64_t>(blockIdx.x) * cols + col] = s;
  }
}

// Rows too long for a block's registers: one value a lane, the rows read twice.  dw
// is summed by columns in a kernel of its own.  (bf16 8192 x 18432 with dh and dw 902 us,
// 1.3 TB/s of what it cannot do without.)
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_long_kernel(const __grid_constant__ NormBwdParams p) {
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
    dot = row_sum(dot, tpr, slots, flip, 0);
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
__global__ void norm_bwd_long_dw_kernel(const __grid_constant__ NormBwdParams p) {
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

// dw[col] = the partial rows' sum: 32 columns a block, and 32 warps that share
// the rows, joined in a fixed order.
__global__ void __launch_bounds__(1024)
    norm_bwd_dw_kernel(const float* partials, int blocks, int32_t cols, float* dw) {
  __shared__ float part[32][33];
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t col = blockIdx.x * 32 + lane;
  ptx::griddep_wait();
  float s = 0.f;
  if (col < cols) {
#pragma unroll 8
    for (int b = warp; b < blocks; b += 32) s += partials[static_cast<int64_t>(b) * cols + col];
  }
  part[warp][lane] = s;
  __syncthreads();
  s = warp_sum(part[lane][warp]);  // column `warp` of the block
  if (lane == 0 && blockIdx.x * 32 + warp < cols) dw[blockIdx.x * 32 + warp] = s;
}

template <typename T, int C, int R>
cudaError_t launch_norm_bwd_r(const NormBwdParams& p, const RowShape& s, int blocks, cudaStream_t st) {
  constexpr size_t smem = static_cast<size_t>(bwd_depth<T, C, R>()) * (kRowThreads / 32) * C * 3 * WarpRow<T>::kBytes;
  const cudaError_t e = allow_smem<norm_bwd_kernel<T, C, R>>();
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_bwd_kernel<T, C, R>, dim3(blocks), dim3(s.per * s.tpr), smem, st, p, s.tpr);
}

template <typename T, int C>
cudaError_t launch_norm_bwd_c(const NormBwdParams& p, int lie, const RowShape& s, int blocks, cudaStream_t st) {
  if (lie == ROWS_ALIGNED) return launch_norm_bwd_r<T, C, ROWS_ALIGNED>(p, s, blocks, st);
  if (lie == ROWS_ALIKE) return launch_norm_bwd_r<T, C, ROWS_ALIKE>(p, s, blocks, st);
  return launch_norm_bwd_r<T, C, ROWS_ANY>(p, s, blocks, st);
}

template <typename T>
cudaError_t launch_norm_bwd_t(const NormBwdParams& p, int sms, cudaStream_t st) {
  int blocks = norm_bwd_blocks(p.rows, sms);
  cudaError_t e;
  if (p.rows == 0) {
    // no rows: dw is zero
  } else if (p.cols <= kMaxCols) {
    int lie = p.rows_lie;
    int64_t chunks = (p.cols + 7) / 8;
    if (lie == ROWS_ALIKE) {
      const int64_t more = alike_chunks(p.cols, sizeof(T));
      if (more * 8 <= kMaxCols && sms >= 8) chunks = more;
      else lie = ROWS_ANY;
    }
    // From 513 chunks on, two a thread leave a block with one row at work and nothing to do
    // while its sum comes together; four leave two or three, but fewer on their way.  In 16
    // bits that is better for three (8000 x 5120 65 to 62 us, 8192 columns 49 to 54), and in
    // ALIKE, where a row's ends take longer (12000 x 4097 108 to 79 us; 1999 columns 70 to 73).
    const bool four = sizeof(T) == 2 && (lie == ROWS_ALIKE || whole_warps(chunks, 4) * 3 <= kRowThreads);
    const RowShape s = many_registers(chunks, four ? kRowThreads : 2 * kRowThreads, p.rows, sms < 64 ? sms : 64);
    const int64_t want = (p.rows + s.per - 1) / s.per;
    if (want < blocks) blocks = static_cast<int>(want);
    if (lie == ROWS_ALIKE) blocks = alike_blocks(p.rows, s.per, blocks);
    e = s.c == 1   ? launch_norm_bwd_c<T, 1>(p, lie, s, blocks, st)
        : s.c == 2 ? launch_norm_bwd_c<T, 2>(p, lie, s, blocks, st)
                   : launch_norm_bwd_c<T, 4>(p, lie, s, blocks, st);
    if (e != cudaSuccess) return e;
  } else {
    // dw first: dx may overwrite dy or h
    if (p.dw != nullptr) {
      e = launch_pdl(norm_bwd_long_dw_kernel<T>, dim3((p.cols + 255) / 256, blocks), dim3(256), 0, st, p);
      if (e != cudaSuccess) return e;
    }
    e = launch_pdl(norm_bwd_long_kernel<T>, dim3(static_cast<unsigned>(p.rows < 65536 ? p.rows : 65536)),
                   dim3(kMaxThreads), 0, st, p);
    if (e != cudaSuccess) return e;
  }
  if (p.dw == nullptr) return cudaSuccess;
  return launch_pdl(norm_bwd_dw_kernel, dim3((p.cols + 31) / 32), dim3(1024), 0, st,
                    static_cast<const float*>(p.partials), blocks, p.cols, p.dw);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, int sms, cudaStream_t st) {
  if (p.dtype == 0) return launch_norm_f<__nv_bfloat16>(p, sms, st);
  if (p.dtype == 1) return launch_norm_f<__half>(p, sms, st);
  return launch_norm_f<float>(p, sms, st);
}

int norm_bwd_blocks(int64_t rows, int sms) {
  return static_cast<int>(rows < sms ? rows : sms);
}

cudaError_t launch_norm_bwd(const NormBwdParams& p, int sms, cudaStream_t st) {
  if (p.dtype == 0) return launch_norm_bwd_t<__nv_bfloat16>(p, sms, st);
  if (p.dtype == 1) return launch_norm_bwd_t<__half>(p, sms, st);
  return launch_norm_bwd_t<float>(p, sms, st);
}

}  // namespace lowp
}  // namespace gge
