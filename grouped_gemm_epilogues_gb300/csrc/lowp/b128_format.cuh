// 8-bit codes with one fp32 scale for each block of 128 columns (of one row, or of 128
// rows): value = code * scale,
//
//   scale = max(amax * (1 / top), 2^-126)      code = round_sat(x * (1 / scale))
//
// top 448 (e4m3) or 57344 (e5m2).  The least scale is the smallest normal number: its
// reciprocal is finite, and a block of zeros needs no case of its own.  A block that holds
// an infinity or a NaN gets a NaN scale.  The product with the rounded 1 / top and the
// correctly rounded reciprocal are the definition, so that codes and scales are the same
// everywhere; a quotient that rounds above top is held to it by the conversion.
#pragma once

#include "mx_format.cuh"

namespace gge {
namespace b128 {

constexpr int kBlock = 128;

// A matrix in this form as the kernels see it.
struct View {
  uint8_t* codes;               // NULL: absent
  float* scales;
  int64_t ld, batch;            // bytes of codes between rows and batches
  int64_t s_row, s_col, s_batch;
  int32_t shift;                // log2 of a block's rows: 0 or 7
  int32_t e5m2;

  __device__ __forceinline__ float* scale(int64_t row, int64_t block, int64_t l) const {
    return scales + (row >> shift) * s_row + block * s_col + l * s_batch;
  }
};

// A block's scale from its largest |x| (as bits), and the factor its values are multiplied
// by before they are rounded.
template <bool E5M2>
__device__ __forceinline__ float block_scale(uint32_t amax_bits, float& factor) {
  constexpr float kInvTop = 1.0f / (E5M2 ? 57344.0f : 448.0f);
  const float s = fmaxf(__uint_as_float(amax_bits) * kInvTop, 1.17549435e-38f);
  const bool bad = amax_bits >= 0x7f800000u;
  factor = bad ? 0.f : __frcp_rn(s);
  return bad ? __uint_as_float(0x7fc00000u) : s;
}

__device__ __forceinline__ uint32_t pack_e5m2x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

template <bool E5M2>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  if constexpr (E5M2) return pack_e5m2x4(a, b, c, d);
  else return mx::pack_e4m3x4(a, b, c, d);
}

// Two codes (the low 16 bits) as numbers.
template <bool E5M2>
__device__ __forceinline__ float2 unpack2(uint32_t two) {
  if constexpr (E5M2) {
    // e5m2 is the upper byte of an fp16 number
    const uint32_t h = __byte_perm(two, 0u, 0x1404);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
  } else {
    return mx::e4m3x2_to_float2(two & 0xffffu);
  }
}

// Four codes times their scale.
template <bool E5M2>
__device__ __forceinline__ void values4(uint32_t w, float unit, float2 (&v)[2]) {
  v[0] = __fmul2_rn(unpack2<E5M2>(w), make_float2(unit, unit));
  v[1] = __fmul2_rn(unpack2<E5M2>(w >> 16), make_float2(unit, unit));
}
template <bool E5M2>
__device__ __forceinline__ void values8(uint2 w, float unit, float2 (&v)[4]) {
  float2 a[2], b[2];
  values4<E5M2>(w.x, unit, a);
  values4<E5M2>(w.y, unit, b);
  v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1];
}
__device__ __forceinline__ void values8_any(bool e5m2, uint2 w, float unit, float2 (&v)[4]) {
  if (e5m2) values8<true>(w, unit, v);
  else values8<false>(w, unit, v);
}

// Eight values times a factor to eight codes.
template <bool E5M2>
__device__ __forceinline__ uint2 codes8(const float2 (&v)[4], float factor) {
  float2 c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = __fmul2_rn(v[i], make_float2(factor, factor));
  return make_uint2(pack4<E5M2>(c[0].x, c[0].y, c[1].x, c[1].y), pack4<E5M2>(c[2].x, c[2].y, c[3].x, c[3].y));
}

// The largest |value| of eight, as bits (a NaN's or an infinity's are above every number's).
__device__ __forceinline__ uint32_t amax8(const float2 (&v)[4]) {
  using mx::max_abs;
  return mx::abs_bits(max_abs(max_abs(max_abs(v[0].x, v[0].y), max_abs(v[1].x, v[1].y)),
                              max_abs(max_abs(v[2].x, v[2].y), max_abs(v[3].x, v[3].y))));
}

// Store the first n of eight codes (n may be 8 or more, or below 1).
__device__ __forceinline__ void store_codes8(uint8_t* p, uint2 w, int32_t n) {
  if (n >= 8) {
    *reinterpret_cast<uint2*>(p) = w;
  } else if (n > 0) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = static_cast<uint8_t>((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
  }
}

// Quantise eight consecutive values a lane, 16 neighbouring lanes to a block (values past a
// row's end are zeros).  Every lane of the warp calls this.
template <bool E5M2>
__device__ __forceinline__ uint2 quantise8(const float2 (&v)[4], float& unit) {
  uint32_t amax = amax8(v);
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  float factor;
  unit = block_scale<E5M2>(amax, factor);
  return codes8<E5M2>(v, factor);
}

}  // namespace b128
}  // namespace gge
