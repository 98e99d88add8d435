// e4m3 numbers and the scales of a paged cache in 8 bits (fa_cache_e4m3.cu,
// fa_decode_e4m3.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fa_paged.cuh"
#include "sm103_ptx.cuh"

namespace fa {

// Two numbers to e4m3, ties to even, `lo` in bits 0-7.  |x| <= 448 and NaN come
// out as such; anything larger would become 448.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  return pack_e4m3x2(a, b) | pack_e4m3x2(c, d) << 16;
}
// Two fp16 numbers to e4m3, in the same way.
__device__ __forceinline__ uint32_t pack_e4m3x2(__half2 x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
  return r;
}
// The numbers in bits 0-15 and in bits 16-31 as two fp16 each, exactly.
__device__ __forceinline__ uint32_t e4m3x2_lo(uint32_t x) {
  uint32_t r;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi(uint32_t x) {
  uint32_t r;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_float2(uint32_t x) {
  return __half22float2(*reinterpret_cast<const __half2*>(&x));
}
__device__ __forceinline__ float4 e4m3x4_to_float4(uint32_t x) {
  const float2 a = f16x2_to_float2(e4m3x2_lo(x)), b = f16x2_to_float2(e4m3x2_hi(x));
  return make_float4(a.x, a.y, b.x, b.y);
}

// Two numbers to e5m2, in the same way, |x| <= 57344; and back: an e5m2 number is the upper byte of an fp16 one.
__device__ __forceinline__ uint32_t pack_e5m2x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_e5m2x2(__half2 x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2(uint32_t x) { return __byte_perm(x, 0, 0x1404); }

// The smallest power of two s with t <= 448 s, 2^-126 at least, for the bits of
// a finite t >= 0.  448 is 1.75 * 2^8: the addition carries into the exponent
// where t's mantissa is above 1.75.
__device__ __forceinline__ float scale_for(uint32_t t) {
  const int e = (int)((t + 0x1fffffu) >> 23) - 8;
  return __uint_as_float((uint32_t)max(e, 1) << 23);
}
// 1 / s of a power of two, 2^-126 to 2^126.
__device__ __forceinline__ float inverse(float s) { return __uint_as_float(0x7f000000u - __float_as_uint(s)); }

// The power of two that weights are in units of, for the largest of them: at or above it, but between kLeastUnit and
// 2^126, so that it has an inverse and 2^11 times that, which is what weights are multiplied by at most, is finite.  Scales
// go from 2^-126 to beyond 2^126: the largest weight is less by up to 2^11 with the smallest, and twice that with the largest.
constexpr float kLeastUnit = 0x1p-115f;
__device__ __forceinline__ float unit_for(float largest) {
  const uint32_t up = (__float_as_uint(fmaxf(largest, kLeastUnit)) + 0x7fffffu) & 0x7f800000u;
  return __uint_as_float(min(up, 0x7e800000u));
}

}  // namespace fa
