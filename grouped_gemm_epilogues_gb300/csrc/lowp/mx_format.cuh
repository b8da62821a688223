// Microscaled number formats: codes, block scales and their layout.
//
//   format   code   block  scale
//   mxfp8    e4m3   32     2^e, one biased exponent byte (255: NaN)
//   mxfp4    e2m1   32     2^e, one biased exponent byte (255: NaN)
//   nvfp4    e2m1   16     e4m3, times one fp32 scale a tensor
//
// Power-of-two scales take the smallest 2^e with amax <= 2^e * (largest code),
// so no value of a block saturates.  With amax = 1.f * 2^k and the largest code
// 1.c * 2^top that is e = k - top, plus one where the fraction f is above c:
// integer arithmetic on the float's bits, and x * 2^-e is exact.  nvfp4 takes
// s = e4m3(max(amax / (6 t), 2^-9)) and codes e2m1(x * (1 / (s t))).  A block
// that holds an infinity or a NaN gets a NaN scale: all its values read back as
// NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

namespace gge {
namespace mx {

enum : int32_t { FMT_MXFP8 = 0, FMT_MXFP4 = 1, FMT_NVFP4 = 2, FMT_NONE = 3 };

template <int FMT>
struct Fmt {
  static constexpr int kBlock = (FMT == FMT_NVFP4) ? 16 : 32;  // values that share a scale
  static constexpr int kBits = (FMT == FMT_MXFP8) ? 8 : 4;
  static constexpr int kGroup = 4 * kBlock;  // values whose scales share a 4-byte word
};

// Scales lie in 512-byte tiles of 128 rows x 4 blocks, tiles of one row block
// consecutive along K.  Inside a tile, row r's four scales are the word at
// (r % 32) * 16 + (r % 128 / 32) * 4: the layout the tensor core's scale operand
// copy (32 lanes x 128 bits) reads.  `kg` is the block index / 4.
__host__ __device__ __forceinline__ int64_t scale_word(int64_t row, int64_t kg, int64_t kgroups) {
  return ((row >> 7) * kgroups + kg) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// Columns up to the end of a row's last scale word (its blocks past the row are padding;
// a row of up to 2^31 columns has up to 2^25 words, so the product takes 64 bits).
template <int FMT>
__host__ __device__ __forceinline__ int64_t scale_span(int64_t kgroups) {
  return kgroups * Fmt<FMT>::kGroup;
}

// ------------------------------------------------------------------ scales

// Biased exponent of a power-of-two scale from a block's largest |x| (as bits).
template <int FMT>
__device__ __forceinline__ uint32_t pow2_scale(uint32_t amax_bits) {
  constexpr int top = (FMT == FMT_MXFP8) ? 8 : 2;                    // 448 = 1.75 * 2^8, 6 = 1.5 * 2^2
  constexpr uint32_t frac = (FMT == FMT_MXFP8) ? 0x600000u : 0x400000u;
  if (amax_bits >= 0x7f800000u) return 255u;
  const int e = static_cast<int>(amax_bits >> 23) + ((amax_bits & 0x7fffffu) > frac ? 1 : 0) - top;
  return static_cast<uint32_t>(max(e, 0));
}

// 2^(e - 127) and 2^(127 - e) for a biased exponent e in [0, 253]
__device__ __forceinline__ float pow2_value(uint32_t e) {
  return __uint_as_float(e == 0u ? 0x400000u : (e == 255u ? 0x7fc00000u : e << 23));
}
__device__ __forceinline__ float pow2_inverse(uint32_t e) {
  return __uint_as_float((254u - e) << 23);
}

// e4m3 code of one non-negative value (round to nearest even, saturating).
__device__ __forceinline__ uint32_t e4m3_of(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ float2 e2m1x2_to_float2(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
      : "=r"(h) : "r"(two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A block's scale: the stored byte, and the factor its values are multiplied
// by before rounding to codes (0 where the block is not finite: its codes are of
// no account then, NaN times anything is NaN).
template <int FMT>
__device__ __forceinline__ uint32_t block_scale(uint32_t amax_bits, float tensor_scale,
                                                float& factor) {
  if constexpr (FMT == FMT_NVFP4) {
    if (amax_bits >= 0x7f800000u) {
      factor = 0.f;
      return 0x7fu;
    }
    const float v = __uint_as_float(amax_bits) / (6.0f * tensor_scale);
    const uint32_t s = e4m3_of(fminf(fmaxf(v, 0.001953125f), 448.0f));
    factor = 1.0f / (e4m3x2_to_float2(s).x * tensor_scale);
    return s;
  } else {
    const uint32_t e = pow2_scale<FMT>(amax_bits);
    factor = e == 255u ? 0.f : pow2_inverse(e);
    return e;
  }
}

// The number a stored scale byte stands for (without the tensor scale).
template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t s) {
  if constexpr (FMT == FMT_NVFP4) return e4m3x2_to_float2(s).x;
  else return pow2_value(s);
}

// ------------------------------------------------------------------- codes

// |x| as bits; the largest of them finds infinities and NaN as well (their bits
// are above every finite value's).
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The larger of |a| and |b|, NaN if either is, with a sign of no meaning.
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Eight values to eight 4-bit codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight scaled values to codes: 8 bytes (two words) or 4 bytes (w.x).
template <int FMT>
__device__ __forceinline__ uint2 pack8(const float (&v)[8]) {
  if constexpr (FMT == FMT_MXFP8)
    return make_uint2(pack_e4m3x4(v[0], v[1], v[2], v[3]), pack_e4m3x4(v[4], v[5], v[6], v[7]));
  else
    return make_uint2(pack_e2m1x8(v), 0u);
}

// ... and back: the code values
template <int FMT>
__device__ __forceinline__ void unpack8(uint2 w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f;
    if constexpr (FMT == FMT_MXFP8) f = e4m3x2_to_float2(((i < 2 ? w.x : w.y) >> (16 * (i & 1))) & 0xffffu);
    else f = e2m1x2_to_float2(w.x >> (8 * i));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// ------------------------------------------------- loads and stores of values

template <typename T> __device__ __forceinline__ float to_float(T x);
template <> __device__ __forceinline__ float to_float(float x) { return x; }
template <> __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }

// Eight consecutive values as they are stored (16 or 32 bytes).
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = r.w[i];
}

// The packed pair of a 16-bit type, and its two values.
template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> { using type = __nv_bfloat162; };
template <> struct Pair<__half> { using type = __half2; };

template <typename T>
__device__ __forceinline__ float2 widen_pair(uint32_t w) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <typename T>
__device__ __forceinline__ uint32_t narrow_pair(float2 v) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// One value of a runtime type (0 bf16, 1 f16, 4 f32: gge_dtype).
__device__ __forceinline__ float load_any(const void* p, int64_t i, int32_t dtype) {
  if (dtype == 0) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  if (dtype == 1) return __half2float(static_cast<const __half*>(p)[i]);
  return static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store_any(void* p, int64_t i, int32_t dtype, float v) {
  if (dtype == 0) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else if (dtype == 1) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else static_cast<float*>(p)[i] = v;
}
// ------------------------------------------------ quantising a warp's chunks

// Where one matrix's codes, scales and (optional) values go.
struct QuantOut {
  uint8_t* codes;
  int64_t ld;        // bytes between rows of codes
  uint8_t* scales;
  int64_t kgroups;   // 4-scale words a row: ceil(blocks / 4)
  const float* tensor_scale;
  void* values;      // NULL: not wanted
  int64_t ldv;
  int32_t v_dtype;
};

// Eight consecutive values as four pairs: the packed fp32 operations take two.
template <typename T>
__device__ __forceinline__ void widen(const Raw8<T>& r, float2 (&v)[4]) {
  if constexpr (sizeof(T) == 4) {
    const float2* f = reinterpret_cast<const float2*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f[i];
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = widen_pair<T>(w[i]);
  }
}

template <typename T>
__device__ __forceinline__ Raw8<T> narrow(const float2 (&v)[4]) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 4) {
    float2* f = reinterpret_cast<float2*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = v[i];
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = narrow_pair<T>(v[i]);
  }
  return r;
}

// round(a + b), value by value.
template <typename T>
__device__ __forceinline__ Raw8<T> add8(const Raw8<T>& a, const Raw8<T>& b) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 4) {
    const float* x = reinterpret_cast<const float*>(&a);
    const float* y = reinterpret_cast<const float*>(&b);
    float* z = reinterpret_cast<float*>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = x[i] + y[i];
  } else {
    using T2 = typename Pair<T>::type;
    const T2* x = reinterpret_cast<const T2*>(&a);
    const T2* y = reinterpret_cast<const T2*>(&b);
    T2* z = reinterpret_cast<T2*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = __hadd2_rn(x[i], y[i]);
  }
  return r;
}

// Eight quantised values of a lane: their codes, their block's scale as a number,
// and, in the first lane of each group of four blocks, the group's scale bytes.
struct Quantised {
  uint2 codes;
  float unit;
  uint32_t word;
};

// Quantise eight consecutive values a lane; neighbouring lanes hold neighbouring
// chunks, four (mx) or two (nvfp4) lanes to a block, and a group of four blocks
// never straddles a warp.  Values past a row's end are zeros; `past`: the lane's
// block lies past the row's last one (its scale byte is padding, 0).  Every lane
// of the warp calls this.
template <int FMT>
__device__ __forceinline__ Quantised quantise8(const float2 (&v)[4], float tensor_scale, bool past) {
  constexpr int kLanes = Fmt<FMT>::kBlock / 8;  // lanes that share a scale
  Quantised r;
  uint32_t amax = abs_bits(max_abs(max_abs(max_abs(v[0].x, v[0].y), max_abs(v[1].x, v[1].y)),
                                   max_abs(max_abs(v[2].x, v[2].y), max_abs(v[3].x, v[3].y))));
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  float factor;
  uint32_t s = block_scale<FMT>(amax, tensor_scale, factor);
  r.unit = scale_value<FMT>(s);
  if (past) s = 0u;
  float c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __fmul2_rn(v[i], make_float2(factor, factor));
    c[2 * i] = f.x;
    c[2 * i + 1] = f.y;
  }
  r.codes = pack8<FMT>(c);
  const uint32_t two = s | (__shfl_down_sync(0xffffffffu, s, kLanes) << 8);
  r.word = two | (__shfl_down_sync(0xffffffffu, two, 2 * kLanes) << 16);
  return r;
}

// Whether this lane is the one that holds its group's scale bytes.
template <int FMT>
__device__ __forceinline__ bool holds_word() {
  return (threadIdx.x & 31) % (Fmt<FMT>::kGroup / 8) == 0;
}

template <int FMT>
__device__ __forceinline__ void store_codes(uint8_t* p, uint2 codes) {
  if constexpr (FMT == FMT_MXFP8) *reinterpret_cast<uint2*>(p) = codes;
  else *reinterpret_cast<uint32_t*>(p) = codes.x;
}

// The numbers that eight codes stand for.
template <int FMT>
__device__ __forceinline__ void code_values(uint2 w, float unit, float tensor_scale, float2 (&v)[4]) {
  float c[8];
  unpack8<FMT>(w, c);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = __fmul2_rn(make_float2(c[2 * i], c[2 * i + 1]), make_float2(unit, unit));
    if constexpr (FMT == FMT_NVFP4) v[i] = __fmul2_rn(v[i], make_float2(tensor_scale, tensor_scale));
  }
}

}  // namespace mx
}  // namespace gge
