// New K and V rows into a paged e4m3 cache with one fp32 scale per page and head.
//
// A page holds P rows of each head.  With A the largest finite |x| of the new rows of a page
// and head, the page's scale becomes
//     s = 2^ceil(log2(A / 448))  (0 for A = 0),   or max(s, s_old) if earlier rows are kept,
// and code = e4m3(x / s), rounded to nearest even; when s > s_old the kept rows are coded
// again, e4m3(decode(code) s_old / s).  A power of two makes both quotients exact (the codes
// lose nothing by it: e4m3 is a floating-point format), so a row coded again keeps its value
// but for results below 2^-6, and rows appended one by one end as rows appended at once.
//
// One CTA per page, head and K or V.  Nothing on the host knows the lengths: CTA slots are
// numbered so that sequence b owns the slots from floor(cu[b] / P) + 2 b on, which leaves it
// at least floor(n / P) + 2 >= the pages its n rows can touch; spare slots exit.  Bound by
// bytes (2 read, 1 written per element) for prompts, by latency for single tokens.
#include <cstdint>

#include "cache.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace attn {
namespace {

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

// x / s: a multiplication when s is a power of two (exact), else the IEEE division.
struct Divisor {
  float s, inv;
  bool pow2;
  __device__ __forceinline__ explicit Divisor(float scale) {
    const uint32_t b = __float_as_uint(scale);
    s = scale;
    pow2 = (b & 0x7fffffu) == 0 && b != 0;             // s >= 2^-126, so 1 / s is normal
    inv = __uint_as_float((254u << 23) - b);
  }
  __device__ __forceinline__ float operator()(float x) const { return pow2 ? x * inv : (s > 0.f ? __fdiv_rn(x, s) : x); }
};

// 8 elements (16 bytes in, 8 bytes out) per thread and step; NV steps cover a page.
template <int D, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) kv_append_kernel(const AppendParams p) {
  __shared__ float red[THREADS / 32];
  const int tid = threadIdx.x;
  // The sequence of this slot: the last b with floor(cu[b] / P) + 2 b <= slot.
  const int slot = blockIdx.x;
  int b = -1;
  bool bad = false;
  for (int base = 0; base < p.B; base += THREADS) {
    const int i = base + tid;
    bool below = false, wrong = false;
    if (i < p.B) {
      const int c0 = p.cu[i], c1 = p.cu[i + 1], len = p.kv_lens[i];
      wrong = c1 < c0 || c0 < 0 || c1 - c0 > len || len > p.max_len || (i == 0 && c0 != 0) ||
              (i == p.B - 1 && c1 != p.total);
      below = c0 / p.page + 2 * i <= slot;
    }
    bad |= __syncthreads_or(wrong) != 0;
    b += __syncthreads_count(below);
  }
  if (bad) {
    if (tid == 0) atomicExch(p.status, DEV_BAD_OFFSETS);
    return;
  }
  const int c0 = p.cu[b], n = p.cu[b + 1] - c0, len = p.kv_lens[b], start = len - n;
  const int blk = start / p.page + slot - (c0 / p.page + 2 * b);
  const int first = blk * p.page;                      // < max_len + 2 pages
  if (n == 0 || first >= len) return;
  const int page = p.table[(long long)b * p.max_pages + blk];
  if (page < 0 || page >= p.num_pages) {
    if (tid == 0) atomicExch(p.status, DEV_BAD_PAGE);
    return;
  }
  const int kept = max(start, first) - first;          // earlier rows of the page
  const int rows = min(len - first, p.page);           // rows in use afterwards
  const int head = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const uint16_t* src = static_cast<const uint16_t*>(is_v ? p.v : p.k) + head * (is_v ? p.v_h : p.k_h);
  const long long st = is_v ? p.v_t : p.k_t;
  const long long ph = (long long)page * p.Hkv + head;
  uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + ph * p.page * D;
  float* scale = (is_v ? p.v_scale : p.k_scale) + ph;

  uint4 x[NV];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (tid + i * THREADS) * 8, r = e / D, c = e % D;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r >= kept && r < rows) x[i] = *reinterpret_cast<const uint4*>(src + (long long)(c0 + first + r - start) * st + c);
    float f[8];
    bf16x8(x[i], f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float a = fabsf(f[k]);
      amax = fmaxf(amax, a < INFINITY ? a : 0.f);      // infinities saturate, NaN stays NaN: neither sets the scale
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((tid & 31) == 0) red[tid >> 5] = amax;
  const float s_old = kept > 0 ? *scale : 0.f;
  __syncthreads();
  amax = red[0];
#pragma unroll
  for (int i = 1; i < THREADS / 32; ++i) amax = fmaxf(amax, red[i]);
  const float s = fmaxf(s_old, pow2_scale(amax));
  if (tid == 0 && s != s_old) *scale = s;
  if (tid == 0 && kept == 0) *scale = s;
  const Divisor div(s);
  const bool again = s > s_old && s_old > 0.f;         // the kept rows' codes change
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (tid + i * THREADS) * 8, r = e / D;
    float f[8];
    if (r < kept) {
      if (!again) continue;
      const uint2 old = *reinterpret_cast<const uint2*>(dst + e);
      e4m3x4_to_f32(old.x, f[0], f[1], f[2], f[3]);
      e4m3x4_to_f32(old.y, f[4], f[5], f[6], f[7]);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = div(f[k] * s_old);
    } else if (r < rows) {
      bf16x8(x[i], f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = div(f[k]);
    } else {
      continue;                                        // rows behind the last one stay as they are
    }
    *reinterpret_cast<uint2*>(dst + e) = e4m3x8(f);
  }
}

template <int D>
cudaError_t launch_d(const AppendParams& p, dim3 grid, cudaStream_t s) {
  const int vecs = p.page * D / 8;                     // 16-byte pieces of a page
  if (vecs == 128) kv_append_kernel<D, 1, 128><<<grid, 128, 0, s>>>(p);
  else if (vecs == 256) kv_append_kernel<D, 1, 256><<<grid, 256, 0, s>>>(p);
  else if (vecs == 512) kv_append_kernel<D, 2, 256><<<grid, 256, 0, s>>>(p);
  else if (vecs == 1024) kv_append_kernel<D, 4, 256><<<grid, 256, 0, s>>>(p);
  else if (vecs == 2048) kv_append_kernel<D, 8, 256><<<grid, 256, 0, s>>>(p);
  else return cudaErrorInvalidValue;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& p, int d, cudaStream_t s) {
  const long long slots = (long long)p.total / p.page + 2LL * p.B;
  if (slots > 0x7fffffffLL || p.Hkv > 65535) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)slots, (unsigned)p.Hkv, 2);
  return d == 64 ? launch_d<64>(p, grid, s) : launch_d<128>(p, grid, s);
}

}  // namespace attn
