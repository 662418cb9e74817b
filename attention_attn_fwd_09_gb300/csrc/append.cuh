// Shared by the kernels that append rows to the paged e4m3 cache (kv_append.cu, rope_append.cu).
#pragma once
#include <cstdint>

#include "cache.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace attn {

// 8 bf16 (one 16-byte load) -> 8 floats
__device__ __forceinline__ void bf16x8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(w[k] << 16);
    f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint2 e4m3x8(const float (&f)[8]) {
  uint32_t h[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(f[2 * k + 1]), "f"(f[2 * k]));
    h[k] = r;
  }
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// 1 / s where that is exact (s a power of two, at least 2^-126, or 0 for rows of zeros), else 0: the
// caller then divides.  Scales that this kernel wrote are powers of two; a cache filled by other
// means may hold others.
__device__ __forceinline__ float exact_inverse(float s) {
  const uint32_t b = __float_as_uint(s);
  if (b == 0) return 1.f;
  return (b & 0x7fffffu) == 0 ? __uint_as_float((254u << 23) - b) : 0.f;
}

// The slot's sequence and page; false: nothing to do (or the offsets are wrong).  Every thread of
// the CTA calls it with the CTA's slot.
struct Slot {
  int kept, rows;            // rows of the page in use before and after
  int first;                 // position of the page's row 0 in its sequence
  int src0;                  // packed row of the page's row 0 (new rows: kept .. rows - 1)
  int page;
};
template <int THREADS>
__device__ __forceinline__ bool find_slot(const AppendParams& p, int slot, Slot& out) {
  const int tid = threadIdx.x;
  // The last b with floor(cu[b] / P) + 2 b <= slot.
  auto look = [&](int i, bool& wrong) -> bool {
    const int c0 = __ldg(p.cu + i), c1 = __ldg(p.cu + i + 1), len = __ldg(p.kv_lens + i);
    wrong |= c1 < c0 || c0 < 0 || c1 - c0 > len || len > p.max_len || (i == 0 && c0 != 0) || (i == p.B - 1 && c1 != p.total);
    return (c0 >> p.page_shift) + 2 * i <= slot;
  };
  bool wrong = false, bad;
  int b = -1;
  if (p.B <= THREADS) {
    bool below = false;
    if (tid < p.B) below = look(tid, wrong);
    bad = __syncthreads_or(wrong) != 0;
    b += __syncthreads_count(below);
  } else {                                   // (several loads under way, one sum: 4096 sequences 85 us, 115 round by round)
    __shared__ int sums[THREADS / 32];
    int below = 0;
#pragma unroll 4
    for (int i = tid; i < p.B; i += THREADS) below += look(i, wrong) ? 1 : 0;
    below = __reduce_add_sync(0xffffffffu, below);
    if ((tid & 31) == 0) sums[tid >> 5] = below;
    bad = __syncthreads_or(wrong) != 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) b += sums[w];
  }
  if (bad) {
    if (tid == 0) atomicExch(p.status, DEV_BAD_OFFSETS);
    return false;
  }
  const int c0 = __ldg(p.cu + b), n = __ldg(p.cu + b + 1) - c0, len = __ldg(p.kv_lens + b), start = len - n;
  const int blk = (start >> p.page_shift) + slot - ((c0 >> p.page_shift) + 2 * b);
  const int first = blk << p.page_shift;                // < max_len + 2 pages
  if (n == 0 || first >= len) return false;
  out.page = __ldg(p.table + (long long)b * p.max_pages + blk);
  if (out.page < 0 || out.page >= p.num_pages) {
    if (tid == 0) atomicExch(p.status, DEV_BAD_PAGE);
    return false;
  }
  out.first = first;
  out.kept = max(start, first) - first;
  out.rows = min(len - first, 1 << p.page_shift);
  out.src0 = c0 + first - start;
  return true;
}

// One head's K or V of a page.
struct Target {
  const uint16_t* src;       // packed row 0 of the head
  long long st;              // token stride
  uint8_t* dst;              // the page's codes
  float* scale;
  __device__ __forceinline__ Target(const AppendParams& p, const Slot& s, int head, bool is_v, int d)
      : src(static_cast<const uint16_t*>(is_v ? p.v : p.k) + head * (is_v ? p.v_h : p.k_h)), st(is_v ? p.v_t : p.k_t) {
    const long long ph = (long long)s.page * p.Hkv + head;
    dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + (ph << p.page_shift) * d;
    scale = (is_v ? p.v_scale : p.k_scale) + ph;
  }
};

// Codes of an earlier row at the page's new scale, which is a power of two (it grew).
__device__ __forceinline__ uint2 recode8(const uint2& old, float s_old, float inv) {
  float f[8];
  e4m3x4_to_f32(old.x, f[0], f[1], f[2], f[3]);
  e4m3x4_to_f32(old.y, f[4], f[5], f[6], f[7]);
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = f[k] * s_old * inv;
  return e4m3x8(f);
}

}  // namespace attn
