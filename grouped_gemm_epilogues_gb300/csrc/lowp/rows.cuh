// Rows that start anywhere, read and written in 16-byte pieces.
//
// A warp's 32 lanes take 8 consecutive values each: 256 columns of a row.  Where
// the row starts `b` bytes past a 16-byte boundary, the aligned pieces that
// cover those columns are one more than a row that starts on one has.  They go
// to shared memory by cp.async (several rows ahead, so that copies stay in
// flight while a row is reduced and written), and each lane puts its 8 values
// together from two neighbouring pieces.  No piece is read past the row's end
// (cp.async takes only the bytes before it); in front of the row a piece holds
// the end of the row before, and in front of the first row single values are
// read.  Writing, the lanes shift their values to the row's boundaries among
// themselves and store whole pieces; only the warp's two ends are single values.
#pragma once

#include "../gge_ptx.cuh"
#include "mx_format.cuh"

namespace gge {
namespace lowp {

using namespace mx;

template <typename T>
struct WarpRow {
  static constexpr int kPieces = sizeof(T) / 2;                  // 16-byte pieces of 8 values
  static constexpr int kBytes = (32 * kPieces + 1) * 16;         // of a warp's 256 columns
};

// N words of a stream, from `b` bytes on (a multiple of 2 below 16).
template <int N>
__device__ __forceinline__ void pick(const uint32_t (&w)[N + 4], uint32_t b, uint32_t (&o)[N]) {
  const bool two = (b & 8u) != 0, one = (b & 4u) != 0;
  const uint32_t half = (b & 2u) * 8;
  uint32_t a[N + 2], c[N + 1];
#pragma unroll
  for (int i = 0; i < N + 2; ++i) a[i] = two ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < N + 1; ++i) c[i] = one ? a[i + 1] : a[i];
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = __funnelshift_r(c[i], c[i + 1], half);
}

// Start copying this warp's 256 columns of a row to `dst`.  `at`: this lane's first
// value, `left`: bytes from there to the row's end (it may be negative).  `first`:
// nothing may be read in front of the row, which starts at this warp's lane 0.
template <typename T>
__device__ __forceinline__ void copy_row(uint32_t dst, const T* at, int32_t left, bool first) {
  constexpr int P = WarpRow<T>::kPieces;
  const int lane = threadIdx.x & 31;
  const int32_t b = static_cast<int32_t>(reinterpret_cast<uintptr_t>(at)) & 15;
  const uint8_t* src = reinterpret_cast<const uint8_t*>(at) - b;  // of the lane's first piece
  left += b;
  dst += 16u * P * lane;
  if (first && b != 0) {  // (the whole warp: one row of a matrix at most)
    if (lane == 0) {
      for (int32_t o = b; o < min(16, left); o += sizeof(T)) {
        if constexpr (sizeof(T) == 2)
          ptx::st_shared_u16(dst + o, *reinterpret_cast<const uint16_t*>(src + o));
        else
          ptx::st_shared_u32(dst + o, *reinterpret_cast<const uint32_t*>(src + o));
      }
    } else if (left > 0) {
      ptx::cp_async_16(dst, src, static_cast<uint32_t>(min(16, left)));
    }
  } else if (left > 0) {
    ptx::cp_async_16(dst, src, static_cast<uint32_t>(min(16, left)));
  }
#pragma unroll
  for (int j = 1; j <= P; ++j)
    if ((j < P || lane == 31) && left > 16 * j)
      ptx::cp_async_16(dst + 16 * j, src + 16 * j, static_cast<uint32_t>(min(16, left - 16 * j)));
}

// A lane's 8 values of a copied row, after the copy has landed (values past the
// row's end are whatever the buffer held).  `b`: the row's offset from a 16-byte
// boundary, the same for every 256 columns of it.
template <typename T>
__device__ __forceinline__ Raw8<T> take_row(uint32_t src, uint32_t b) {
  constexpr int P = WarpRow<T>::kPieces;
  const int lane = threadIdx.x & 31;
  uint32_t w[4 * P + 4];
#pragma unroll
  for (int j = 0; j <= P; ++j) {
    const uint4 v = ptx::ld_shared_v4(src + 16u * (lane * P + j));
    w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
  }
  uint32_t o[4 * P];
  pick(w, b, o);
  Raw8<T> r;
#pragma unroll
  for (int j = 0; j < P; ++j) r.w[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
  return r;
}

// The same straight from global memory, for a lane on its own: columns [col, col
// + 8) of the row at `row`; values past its end are zero.  Reads whole pieces
// inside [lo, row end) only.
template <typename T>
__device__ __forceinline__ Raw8<T> load_row8(const T* row, int32_t col, int32_t cols, const T* lo) {
  constexpr int P = WarpRow<T>::kPieces;
  const uintptr_t at = reinterpret_cast<uintptr_t>(row + col);
  const uint32_t b = static_cast<uint32_t>(at) & 15u;
  Raw8<T> r;
  if (b == 0 && col + 8 <= cols) return load8(row + col);
  const uintptr_t piece0 = at - b;
  const uintptr_t end = reinterpret_cast<uintptr_t>(row + cols);
  if (b != 0 && piece0 >= reinterpret_cast<uintptr_t>(lo) && piece0 + 16u * (P + 1) <= end) {
    uint32_t w[4 * P + 4];
#pragma unroll
    for (int j = 0; j <= P; ++j) {
      const uint4 v = *reinterpret_cast<const uint4*>(piece0 + 16u * j);
      w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
    }
    uint32_t o[4 * P];
    pick(w, b, o);
#pragma unroll
    for (int j = 0; j < P; ++j) r.w[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
    return r;
  }
  T* t = reinterpret_cast<T*>(&r);
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = col + i < cols ? row[col + i] : from_float<T>(0.f);
  return r;
}

// Values k to 7 of the 8 that belong at `at`, a 16-byte boundary; the first n of them.
template <typename T>
__device__ __forceinline__ void store_from(T* at, int32_t k, const Raw8<T>& v) {
  if constexpr (sizeof(T) == 2) {
    const uint4 w = v.w[0];
    uint8_t* b = reinterpret_cast<uint8_t*>(at);
    if (k & 1) {
      const uint32_t x = (k & 4) ? ((k & 2) ? w.w : w.z) : ((k & 2) ? w.y : w.x);
      *reinterpret_cast<uint16_t*>(b + 2 * k) = static_cast<uint16_t>(x >> 16);
    }
    const int32_t e = (k + 1) & ~1;  // 0, 2, .. 8
    if (e & 2) *reinterpret_cast<uint32_t*>(b + 2 * e) = (e & 4) ? w.w : w.y;
    if (e <= 4) {
      *reinterpret_cast<uint2*>(b + 8) = make_uint2(w.z, w.w);
      if (e == 0) *reinterpret_cast<uint2*>(b) = make_uint2(w.x, w.y);
    }
  } else {
    const T* t = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= k) at[i] = t[i];
  }
}
template <typename T>
__device__ __forceinline__ void store_up_to(T* at, int32_t n, const Raw8<T>& v) {
  if constexpr (sizeof(T) == 2) {
    const uint4 w = v.w[0];
    uint8_t* b = reinterpret_cast<uint8_t*>(at);
    if (n & 4) *reinterpret_cast<uint2*>(b) = make_uint2(w.x, w.y);
    if (n & 2) *reinterpret_cast<uint32_t*>(b + 2 * (n & 4)) = (n & 4) ? w.z : w.x;
    if (n & 1) {
      const uint32_t x = (n & 4) ? ((n & 2) ? w.w : w.z) : ((n & 2) ? w.y : w.x);
      *reinterpret_cast<uint16_t*>(b + 2 * (n & 6)) = static_cast<uint16_t>(x);
    }
  } else {
    const T* t = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) at[i] = t[i];
  }
}

// Eight values in 16-byte pieces where the row allows it, for a lane on its own.
template <typename T>
__device__ __forceinline__ void store_row8_aligned(T* row, int32_t col, int32_t cols, const Raw8<T>& v) {
  if (col + 8 <= cols) {
    store8(row + col, v);
  } else if (col < cols) {
    store_up_to(row + col, cols - col, v);
  }
}

// Store 8 values a lane to columns [col, col + 8) of the row at `row`; columns >=
// cols are not written.  Warp-collective.
template <typename T>
__device__ __forceinline__ void store_row8(T* row, int32_t col, int32_t cols, const Raw8<T>& v) {
  constexpr int P = WarpRow<T>::kPieces;
  const int lane = threadIdx.x & 31;
  const uint32_t b = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row)) & 15u;
  if (b == 0) {  // (col is a multiple of 8)
    store_row8_aligned(row, col, cols, v);
    return;
  }
  // Shifted by k columns, 8 values start on the boundary: the previous lane's last
  // k and this lane's first 8 - k.  The warp's first 8 - k and last k are left over.
  const int32_t k = static_cast<int32_t>(b / sizeof(T));
  const int32_t start = col - k;
  uint32_t w[4 * P + 4], o[4 * P];
#pragma unroll
  for (int j = 0; j < P; ++j)
    w[4 + 4 * j] = v.w[j].x, w[5 + 4 * j] = v.w[j].y, w[6 + 4 * j] = v.w[j].z, w[7 + 4 * j] = v.w[j].w;
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = __shfl_up_sync(0xffffffffu, w[4 * P + j], 1);  // its last piece
  pick(w, 16u - b, o);
  if (lane > 0 && start + 8 <= cols) {
    Raw8<T> r;
#pragma unroll
    for (int j = 0; j < P; ++j) r.w[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
    store8(row + start, r);
  } else if (lane > 0) {  // the row's end
    const T* s = reinterpret_cast<const T*>(o);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (start + i < cols) row[start + i] = s[i];
  }
  // lanes 0-7 store the left-over values, one each
  const int i = lane & 7;
  const bool front = i < 8 - k;
  uint32_t left = 0u;
#pragma unroll
  for (int j = 0; j < 4 * P; ++j) {
    const uint32_t x = __shfl_sync(0xffffffffu, w[4 + j], front ? 0 : 31);
    if ((P == 1 ? i >> 1 : i) == j) left = x;
  }
  const int32_t c = col - lane * 8 + (front ? 0 : 31 * 8) + i;
  if (lane < 8 && c < cols) {
    if constexpr (P == 1)
      reinterpret_cast<uint16_t*>(row)[c] = static_cast<uint16_t>((i & 1) ? left >> 16 : left);
    else
      reinterpret_cast<uint32_t*>(row)[c] = left;
  }
}

// ... of a runtime type (0 bf16, 1 f16, 4 f32: gge_dtype), at element `at` of
// `base`; AL: the rows start on 16-byte boundaries.
template <bool AL, typename T>
__device__ __forceinline__ void store_row8_t(void* base, int64_t at, int32_t col, int32_t cols,
                                             const float2 (&v)[4]) {
  T* row = static_cast<T*>(base) + at;
  if constexpr (AL) store_row8_aligned(row, col, cols, narrow<T>(v));
  else store_row8(row, col, cols, narrow<T>(v));
}
template <bool AL>
__device__ __forceinline__ void store_row8_any(void* base, int64_t at, int32_t dtype, int32_t col,
                                               int32_t cols, const float2 (&v)[4]) {
  if (dtype == 0) store_row8_t<AL, __nv_bfloat16>(base, at, col, cols, v);
  else if (dtype == 1) store_row8_t<AL, __half>(base, at, col, cols, v);
  else store_row8_t<AL, float>(base, at, col, cols, v);
}

template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

}  // namespace lowp
}  // namespace gge
