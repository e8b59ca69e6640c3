// e4m3.hpp -- e4m3 codes under power-of-two scales: the scale that a largest magnitude needs, and the conversions.
#pragma once

#include "common.hpp"

namespace lora {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Exponent bytes that a scale may take: 2^-117 .. 2^120.
constexpr int kExpMin = 10, kExpMax = 247;

// Four values of a row as f32, from registers.
template <typename T>
struct Raw4;
template <>
struct Raw4<float> {
  uint4 r;
  __device__ void load(const float *p) { r = ldg16(p); }
  __device__ void zero() { r = z4(); }
  __device__ float at(int i) const { return __uint_as_float(i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w); }
};
template <>
struct Raw4<u16> {
  uint2 r;
  __device__ void load(const u16 *p) {
    typedef unsigned u32x2n __attribute__((ext_vector_type(2)));
    const u32x2n v = *(const __attribute__((address_space(1))) u32x2n *)(uintptr_t)p;
    r = make_uint2(v.x, v.y);
  }
  __device__ void zero() { r = make_uint2(0u, 0u); }
  __device__ float at(int i) const {
    const uint32_t w = i < 2 ? r.x : r.y;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
};

// Two f32 as bf16, rounded to nearest even, by one instruction (f2bf takes five for each).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// |x|'s bits where x is finite, 0 elsewhere: unsigned order is magnitude order.
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}

// The exponent byte for a largest magnitude m 2^(E - 127), 1 <= m < 2: 448 is
// 1.75 2^8, so 2^(E - 135) does where m <= 1.75 and twice that elsewhere.
__device__ __forceinline__ int exp_for(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u);
  return min(max(e, kExpMin), kExpMax);
}

// Four scaled values as codes; infinities and NaN become NaN, so that they
// show in what reads them.  The conversion rounds to nearest, ties to even,
// and nothing exceeds 448.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv) {
  const float qnan = __uint_as_float(0x7fc00000u);
  a = __builtin_isfinite(a) ? a * inv : qnan;
  b = __builtin_isfinite(b) ? b * inv : qnan;
  c = __builtin_isfinite(c) ? c * inv : qnan;
  d = __builtin_isfinite(d) ? d * inv : qnan;
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

}  // namespace lora
