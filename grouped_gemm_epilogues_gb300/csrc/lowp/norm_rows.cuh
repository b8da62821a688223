// What the kernels that normalise rows share: rows on their way through shared memory, sums
// over the threads of a row, and how rows are spread over a launch's threads.
#pragma once

#include <numeric>

#include "lowp_launch.h"
#include "rows.cuh"

namespace gge {
namespace lowp {

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
inline int alike_blocks(int64_t rows, int per_block, int64_t blocks) {
  if (rows <= blocks * per_block) return static_cast<int>(blocks);
  const int unit = 8 / std::gcd(8, per_block);
  return static_cast<int>(blocks / unit * unit);
}

// How a row is spread: chunks a thread, threads a row (whole warps), rows a block, and
// blocks an SM.  Row groups of several warps have a barrier each, of the 15 beside the
// block's.
struct RowShape {
  int c, tpr, per, blocks;
};
inline int whole_warps(int64_t chunks, int c) { return static_cast<int>((chunks + 32 * c - 1) / (32 * c) * 32); }

// ... with up to 64 registers a thread: blocks such that as many rows as possible are at
// work.  An SM has four quarters of 8 such warps, and a block's warps go round them.
// (1536 columns, 96 threads a row: 5 rows a block, twice, 34 us for 48 M values; 2 rows
// a block, which leaves room for four blocks, 46.)  Few rows have one chunk a thread
// (latency); many two, so that a row's barrier costs less.
inline RowShape many_threads(int64_t chunks, bool few) {
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
inline RowShape many_registers(int64_t chunks, int64_t two, int64_t rows, int spread) {
  const bool few = rows <= spread;
  RowShape s{chunks > (few ? 2 * kRowThreads : two) ? 4 : (chunks > (few ? kRowThreads : 32) ? 2 : 1), 0, 0, 1};
  s.tpr = whole_warps(chunks, s.c);
  s.per = kRowThreads / s.tpr;
  const int64_t each = (rows + spread - 1) / spread;
  if (each < s.per) s.per = static_cast<int>(each);
  return s;
}

// Chunks of a row of `cols` values that starts at any skew.
inline int64_t alike_chunks(int64_t cols, int value_bytes) { return (cols + 16 / value_bytes - 1 + 7) / 8; }

}  // namespace lowp
}  // namespace gge
