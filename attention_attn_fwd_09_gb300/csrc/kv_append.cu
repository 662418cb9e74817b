// New K and V rows into a paged e4m3 cache with one fp32 scale per page and head.
//
// A page holds P rows of each head.  With A the largest finite |x| of the new rows of a page
// and head, the page's scale becomes
//     s = 2^ceil(log2(A / 448))  (0 for A = 0),   or max(s, s_old) if earlier rows are kept,
// and code = e4m3(x / s), rounded to nearest even; when s > s_old the kept rows are coded
// again, e4m3(decode(code) s_old / s).  A power of two makes both quotients exact (the codes
// lose nothing by it: e4m3 is a floating-point format), so a row coded again keeps its value
// but for results below 2^-6, and rows appended one by one end as rows appended at once.  (s_old = 0
// too: rows that read 0, infinities among them, keep reading 0, and NaN stays NaN.)
//
// Nothing on the host knows the lengths: slots are numbered so that sequence b owns the slots
// from floor(cu[b] / P) + 2 b on, which leaves it at least floor(n / P) + 2 >= the pages its n
// rows can touch; spare slots exit.  Two kernels:
//   * prompts (bound by bytes, 2 read and 1 written per element): a CTA per slot, head and K or
//     V holds the page's new rows in registers between the maximum and the rounding, one pass
//     over the data.  8192 rows of 8 heads twice, d = 128: 20.5 us from memory, 4.9
//     TB/s (again and again on rows that L2 holds 15.1; d = 64 9.2);
//   * a few rows per sequence or page (bound by latency): a warp per slot, head and K or V, no
//     barrier behind the search for the slot.  One row of 64 sequences: 2.5 us in a graph.
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

// Largest finite magnitude of bf16 values, as bf16 bits: infinities saturate and NaN stays NaN when
// coded, neither sets the scale.  Two values at a time; bits of infinities and NaN are the largest
// and are looked at again only if they occur.
struct Largest {
  uint32_t two = 0;
  __device__ __forceinline__ void add(const uint4& v) {
    two = __vmaxu2(two, v.x & 0x7fff7fffu);
    two = __vmaxu2(two, v.y & 0x7fff7fffu);
    two = __vmaxu2(two, v.z & 0x7fff7fffu);
    two = __vmaxu2(two, v.w & 0x7fff7fffu);
  }
  __device__ __forceinline__ uint32_t bits() const { return max(two & 0xffffu, two >> 16); }
};
__device__ __noinline__ uint32_t largest_finite(uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  const uint32_t u[4] = {x, y, z, w};
  uint32_t m = 0;
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = u[i >> 1] >> (i & 1) * 16 & 0x7fffu;
    if (a < 0x7f80u) m = max(m, a);
  }
  return m;
}
__device__ __forceinline__ uint2 code8(const uint4& v, float inv) {
  float f[8];
  bf16x8(v, f);
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] *= inv;
  return e4m3x8(f);
}
// The same by division.
__device__ __noinline__ uint2 code8_div(uint4 v, float s) {
  float f[8];
  bf16x8(v, f);
  for (int k = 0; k < 8; ++k) f[k] = __fdiv_rn(f[k], s);
  return e4m3x8(f);
}
// Codes of an earlier row at the page's new scale, which is a power of two (it grew).
__device__ __forceinline__ uint2 recode8(const uint2& old, float s_old, float inv) {
  float f[8];
  e4m3x4_to_f32(old.x, f[0], f[1], f[2], f[3]);
  e4m3x4_to_f32(old.y, f[4], f[5], f[6], f[7]);
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = f[k] * s_old * inv;
  return e4m3x8(f);
}

// 8 elements (16 bytes in, 8 bytes out) per thread and step; NV steps cover a page of one head.
template <int D, int NV, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) kv_append_kernel(const AppendParams p) {
  __shared__ uint32_t red[THREADS / 32];
  constexpr int RPS = THREADS * 8 / D;                 // rows per step
  const int tid = threadIdx.x;
  Slot s;
  if (!find_slot<THREADS>(p, blockIdx.x, s)) return;
  const Target t(p, s, blockIdx.y, blockIdx.z != 0, D);
  const int r0 = tid / (D / 8), c = tid % (D / 8) * 8;
  const float s_old = s.kept > 0 ? *t.scale : 0.f;
  uint4 x[NV];
  const uint16_t* src = t.src + (s.src0 + r0) * t.st + c;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r0 + i * RPS >= s.kept && r0 + i * RPS < s.rows) x[i] = __ldcs(reinterpret_cast<const uint4*>(src));
    src += RPS * t.st;
  }
  Largest big;
#pragma unroll
  for (int i = 0; i < NV; ++i) big.add(x[i]);
  uint32_t amax = big.bits();
  if (amax >= 0x7f80u) {
    amax = 0;
#pragma unroll 1
    for (int i = 0; i < NV; ++i) {
      uint4 v = x[0];
#pragma unroll
      for (int k = 1; k < NV; ++k)
        if (i == k) v = x[k];
      amax = max(amax, largest_finite(v.x, v.y, v.z, v.w));
    }
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  if ((tid & 31) == 0) red[tid >> 5] = amax;
  __syncthreads();
  amax = red[0];
#pragma unroll
  for (int i = 1; i < THREADS / 32; ++i) amax = max(amax, red[i]);
  const float sc = fmaxf(s_old, pow2_scale(__uint_as_float(amax << 16)));
  if (tid == 0) *t.scale = sc;
  const float inv = exact_inverse(sc);
  uint2* out = reinterpret_cast<uint2*>(t.dst + tid * 8);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int r = r0 + i * RPS;                        // rows behind the last one stay as they are
    if (r >= s.kept && r < s.rows) out[i * THREADS] = inv != 0.f ? code8(x[i], inv) : code8_div(x[i], sc);
  }
  if (sc > s_old) {                                    // the kept rows' codes change (under a scale of 0: to 0)
#pragma unroll 1
    for (int i = 0; i < NV && r0 + i * RPS < s.kept; ++i) out[i * THREADS] = recode8(out[i * THREADS], s_old, inv);
  }
}

constexpr int kStepWarps = 8;

// Warp w of block (x, y): head 8 y + w of slot x / 2, K or V by x & 1.
template <int D>
__global__ void __launch_bounds__(kStepWarps * 32) kv_append_step_kernel(const AppendParams p) {
  const int lane = threadIdx.x & 31, head = blockIdx.y * kStepWarps + (threadIdx.x >> 5);
  Slot s;
  if (!find_slot<kStepWarps * 32>(p, blockIdx.x >> 1, s) || head >= p.Hkv) return;
  const Target t(p, s, head, blockIdx.x & 1, D);
  constexpr int RPW = 32 / (D / 8);                    // rows a warp reads at once
  const int r0 = lane / (D / 8), c = lane % (D / 8) * 8;
  const float s_old = s.kept > 0 ? *t.scale : 0.f;
  auto row_of = [&](int r) -> uint4 { return *reinterpret_cast<const uint4*>(t.src + (s.src0 + r) * t.st + c); };
  // (No calls in these loops: they would keep the loads of a page with many new rows from overlapping.)
  uint4 x = make_uint4(0u, 0u, 0u, 0u);
  Largest big;
#pragma unroll 8
  for (int r = s.kept + r0; r < s.rows; r += RPW) {
    x = row_of(r);
    big.add(x);
  }
  uint32_t amax = big.bits();
  if (amax >= 0x7f80u) {
    amax = 0;
    for (int r = s.kept + r0; r < s.rows; r += RPW) {
      const uint4 y = row_of(r);
      amax = max(amax, largest_finite(y.x, y.y, y.z, y.w));
    }
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  const float sc = fmaxf(s_old, pow2_scale(__uint_as_float(amax << 16)));
  const float inv = exact_inverse(sc);
  if (inv != 0.f && s.rows - s.kept <= RPW) {
    if (s.kept + r0 < s.rows) *reinterpret_cast<uint2*>(t.dst + (s.kept + r0) * D + c) = code8(x, inv);
  } else if (inv != 0.f) {
#pragma unroll 8
    for (int r = s.kept + r0; r < s.rows; r += RPW) *reinterpret_cast<uint2*>(t.dst + r * D + c) = code8(row_of(r), inv);
  } else {
    for (int r = s.kept + r0; r < s.rows; r += RPW) *reinterpret_cast<uint2*>(t.dst + r * D + c) = code8_div(row_of(r), sc);
  }
  if (sc > s_old) {
    for (int r = r0; r < s.kept; r += RPW) {
      uint2* out = reinterpret_cast<uint2*>(t.dst + r * D + c);
      *out = recode8(*out, s_old, inv);
    }
  }
  __syncwarp();                                        // every lane has read the old scale
  if (lane == 0) *t.scale = sc;
}

template <int D>
cudaError_t launch_d(const AppendParams& p, dim3 grid, cudaStream_t s) {
  const int vecs = p.page * D / 8;                     // 16-byte pieces of a page
  if (vecs == 128) kv_append_kernel<D, 1, 128, 12><<<grid, 128, 0, s>>>(p);
  else if (vecs == 256) kv_append_kernel<D, 1, 256, 6><<<grid, 256, 0, s>>>(p);
  else if (vecs == 512) kv_append_kernel<D, 2, 256, 6><<<grid, 256, 0, s>>>(p);
  else if (vecs == 1024) kv_append_kernel<D, 4, 256, 5><<<grid, 256, 0, s>>>(p);
  else if (vecs == 2048) kv_append_kernel<D, 8, 256, 4><<<grid, 256, 0, s>>>(p);
  else return cudaErrorInvalidValue;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(AppendParams p, int d, int sms, cudaStream_t s) {
  p.page_shift = p.page == 16 ? 4 : p.page == 32 ? 5 : p.page == 64 ? 6 : 7;
  const long long slots = (long long)p.total / p.page + 2LL * p.B;
  if (slots > 0x3fffffffLL || p.Hkv > 65535) return cudaErrorInvalidValue;
  // Up to 4 rows per sequence on average: a warp per page and head (64 sequences, 8 heads, pages of 128:
  // 1 row each 2.8 us against 7.0 with a CTA each, 4 rows 3.2 against 7.1; a piece of 128 rows among 63
  // single ones, which the host cannot tell from 3 rows each, 9.8 against 7.2).
  // So too many pages with up to 32 new rows on average, a CTA each of which comes and goes for little:
  // 256 pieces of 16 rows 7.5 us against 21.5 (pages of 64: 7.6 against 17.6), 2 x 4096 rows of 8 heads,
  // d = 128, over pages of 16 9.7 against 18.2, of 32 9.5 against 11.9.  Fewer CTAs would leave SMs idle
  // (2 heads, 14 CTAs per SM, 6.2 against 6.1; 1 head, 5.6 against 3.8), more rows are read at one go by
  // a CTA (4 x 8192 over pages of 64 33 against 61 with a warp each).
  const bool small = p.total <= 32 * slots && 2 * slots * p.Hkv >= 16LL * sms;
  if (p.total <= 4LL * p.B || small) {
    const dim3 grid((unsigned)(2 * slots), (unsigned)((p.Hkv + kStepWarps - 1) / kStepWarps));
    if (d == 64) kv_append_step_kernel<64><<<grid, kStepWarps * 32, 0, s>>>(p);
    else kv_append_step_kernel<128><<<grid, kStepWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
  }
  const dim3 grid((unsigned)slots, (unsigned)p.Hkv, 2);
  return d == 64 ? launch_d<64>(p, grid, s) : launch_d<128>(p, grid, s);
}

}  // namespace attn
