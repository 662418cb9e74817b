// Shared by the kernels of the paged e4m3 cache: number formats, the workspace of partial results.
#pragma once
#include <cstdint>

#include <cuda_fp16.h>

#include "kernels.h"

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

constexpr float kMinScale = 1.17549435e-38f;   // 2^-126: a reference for V scales that never is 0
constexpr float kLn2 = 0.6931471805599453f;

// Attention over the cache cuts its work evenly by keys, so a unit (some query rows of one
// sequence and K/V head) may be worked on by several CTAs, each of which leaves a partial
// result: per row m (running maximum, log2), l (sum of 2^(s - m)), a reference scale r and
// O / r.  A CTA has at most two: partial 0 for its first unit, partial 1 for its last.
// Workspace: per CTA an int4 {K/V head, first packed query, queries, 2 x further CTAs + which
// partial} for the unit that starts in it and is cut (last field < 2: none); then per partial and
// row (m, l, r, -); then per partial the O rows as [d / 4][rows] pieces of 4 columns.
struct CacheWs {
  size_t stat, part, total;
};
__host__ __device__ inline CacheWs cache_ws(int ctas, int rows, int d) {
  CacheWs w;
  w.stat = ((size_t)ctas * 16 + 255) & ~size_t(255);
  w.part = w.stat + (((size_t)ctas * 2 * rows * 16 + 255) & ~size_t(255));
  w.total = w.part + (size_t)ctas * 2 * rows * d * 4;
  return w;
}

// NaN codes of V.  A weight of 0 does not silence them (0 NaN = NaN), so a key that only some of a
// tile's queries see must not hold any: its NaN codes are set to 0 where they lie in shared memory,
// and per column the first such key is noted.  A query sees the keys up to its own limit, so exactly
// the queries whose limit lies behind the noted key are NaN in that column.
__device__ __forceinline__ bool any_nan_code(const uint4& v) {
  const uint32_t a = (v.x & 0x7f7f7f7fu) + 0x01010101u, b = (v.y & 0x7f7f7f7fu) + 0x01010101u;
  const uint32_t c = (v.z & 0x7f7f7f7fu) + 0x01010101u, d = (v.w & 0x7f7f7f7fu) + 0x01010101u;
  return ((a | b | c | d) & 0x80808080u) != 0;
}
// first[0 .. 15]: of the piece's 16 columns.
__device__ __forceinline__ void take_nan_codes(uint8_t* piece, int key, int* first, int* any) {
#pragma unroll 1
  for (int i = 0; i < 16; ++i) {
    if ((piece[i] & 0x7f) != 0x7f) continue;
    piece[i] = 0;
    atomicMin(first + i, key);
    *any = 1;
  }
}
constexpr int kNoKey = 0x7fffffff;

// How long a CTA that gives up waits for its own copies and products in flight: not less than 10 ms,
// however short a wait may be.
__device__ __forceinline__ unsigned long long drain_ns(const CacheParams& p) { return max(p.wait_ns, 10000000ull); }

}  // namespace attn
