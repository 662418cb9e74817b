// Shared by the kernels of the paged e4m3 cache: number formats.
#pragma once
#include <cstdint>

#include <cuda_fp16.h>

namespace attn {

// Two e4m3 codes (low byte -> low half) as f16, exact.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t pair) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(pair));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2_hi(uint32_t quad) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(quad));
  return r;
}
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t quad, float& a, float& b, float& c, float& d) {
  const uint32_t lo = e4m3x2_f16x2(quad), hi = e4m3x2_f16x2_hi(quad);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  a = x.x; b = x.y; c = y.x; d = y.y;
}

// 2^ceil(log2(amax / 448)), the smallest power of two with amax / s <= 448: amax = m 2^e with
// 1 <= m < 2 and 448 = 1.75 * 2^8.  0 for amax = 0; never below 2^-126, so that 1 / s is normal.
__device__ __forceinline__ float pow2_scale(float amax) {
  if (!(amax > 0.f)) return 0.f;
  const uint32_t bits = __float_as_uint(amax);
  const int e = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)max(e, 1) << 23);
}

}  // namespace attn
