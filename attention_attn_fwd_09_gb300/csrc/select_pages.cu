// The pages of a paged e4m3 cache that each query is to read, by an upper bound of its scores there.
//
// A page's bounds hold its smallest and largest code per column (lo, hi).  No key of the page can
// score more against q than
//     s(q, page) = scale_page sum_c max(q_c, 0) hi_c + min(q_c, 0) lo_c,
// and the heads of a group, which share a list, go by the largest of theirs.  The first pages (which
// much attention falls on whatever the query) and the last ones (the nearest keys) are always
// listed, the best of the others fill the list, ascending; a sequence with few enough pages lists all.
//
// What is chosen is what exact scores choose (equal ones by number), whatever order a sum is taken
// in: the kernels score in fp32 with a bound on their error, and only pages too near the border to
// tell are scored again in 64 bits.  So the list depends on nothing but the query and the bounds.
//
// Two dependent launches:
//   * scores, bound by the bounds' bytes (2 d per page and K/V head): a warp takes 8 pages as the
//     columns of mma.m16n8k16, the rows are queries x heads of a group (as in fwd_cache.cu), the
//     products run over [max(q, 0), min(q, 0)] against [hi, lo].  f16 holds the codes and, scaled by a power
//     of two per row, q (exact down to 2^-31 of the row's largest component, off by 2^-39 of it below);
//   * choice, bound by latency: a CTA per query and K/V head bisects for the border.
#include <cstdint>
#include <mutex>

#include "cache.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;
constexpr int kStepPages = kSelWarps * 8;    // pages that a CTA scores at once
constexpr float kBig = 3.0e38f;

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t positive(uint32_t x) {
  const __half2 z = __float2half2_rn(0.f), r = __hmax2(*reinterpret_cast<const __half2*>(&x), z);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t negative(uint32_t x) {
  const __half2 z = __float2half2_rn(0.f), r = __hmin2(*reinterpret_cast<const __half2*>(&x), z);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Where a tile of queries stands.
struct Tile {
  int b, q0, n, len;         // sequence, its first packed query, queries, keys
};
// The sequence of `slot`, the last one with first slot cu[b] / qn (+ b, when qn > 1) <= slot; false where the
// offsets or lengths are wrong.  All threads of the CTA.
__device__ __forceinline__ bool find_tile(const SelectParams& p, int slot, Tile& out) {
  __shared__ int below;
  bool wrong = false;
  int mine = 0;
  if (threadIdx.x == 0) below = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.B; i += kSelThreads) {
    const int c0 = __ldg(p.cu_q + i), c1 = __ldg(p.cu_q + i + 1), len = __ldg(p.kv_lens + i), n = c1 - c0;
    wrong |= c0 < 0 || c1 < c0 || n > p.max_q || len < 0 || len > p.max_len || (p.causal && n > len) ||
             (i == 0 && c0 != 0) || (i == p.B - 1 && c1 != p.total_q);
    mine += (p.qn > 1 ? c0 / p.qn + i : c0) <= slot ? 1 : 0;
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  if ((threadIdx.x & 31) == 0) atomicAdd(&below, mine);
  if (__syncthreads_or(wrong)) {
    if (threadIdx.x == 0) atomicExch(p.status, DEV_BAD_OFFSETS);
    return false;
  }
  out.b = below - 1;
  out.q0 = __ldg(p.cu_q + out.b);
  out.n = __ldg(p.cu_q + out.b + 1) - out.q0;
  out.len = __ldg(p.kv_lens + out.b);
  return true;
}
// Pages that query i of the sequence sees.
__device__ __forceinline__ int pages_seen(const SelectParams& p, const Tile& t, int i) {
  const int keys = p.causal ? t.len - t.n + i + 1 : t.len;
  return (keys + p.page - 1) >> p.page_shift;
}

// Block: (tile slot, K/V head, chunk of p.chunk pages).  Writes scores [K/V head][query][max_pages] and,
// per chunk, a bound on their error.
template <int D>
__global__ void __launch_bounds__(kSelThreads) select_score_kernel(const SelectParams p) {
  constexpr int KS = D / 16;                 // products of 16 columns
  __shared__ float sums[kSelWarps][16][9];
  __shared__ float norms[16], scale_max[kSelWarps];
  pdl_wait();                                // nothing of global memory before this
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = lane & 3, rq = lane >> 2;
  const int chunk = blockIdx.x % p.chunks, unit = blockIdx.x / p.chunks, h = unit % p.Hkv, slot = unit / p.Hkv;
  Tile t;
  if (!find_tile(p, slot, t)) return;
  // Queries i0 .. i1 - 1 of the sequence.
  const int i0 = p.qn > 1 ? (slot - (t.q0 / p.qn + t.b)) * p.qn : slot - t.q0, i1 = min(i0 + p.qn, t.n);
  if (i0 >= i1) return;                      // a spare slot
  const int seen = pages_seen(p, t, i1 - 1);
  const int begin = max(p.first, chunk * p.chunk), end = min(seen - p.last, (chunk + 1) * p.chunk);
  if (seen <= p.count || begin >= end) return;
  const int* table = p.table + (long long)t.b * p.max_pages;
  const int tiles = p.g > 16 ? (p.g + 15) / 16 : 1;                // of 16 heads, when a group has more
  if (tid < 16) norms[tid] = 0.f;
  float big = 0.f;
  for (int rt = 0; rt < tiles; ++rt) {
    const int heads = min(p.g - rt * 16, 16), rows = tiles > 1 ? heads : (i1 - i0) * p.g;
    // ---- Q: row r is query r / g, head r % g.  As in fwd_cache.cu a thread's columns are 16 neighbouring ones.
    uint32_t qp[KS][4], qm[KS][4];
    float unscale[2];
    __syncthreads();                         // norms
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = rq + 8 * i, qi = tiles > 1 ? 0 : r / p.g, hd = tiles > 1 ? rt * 16 + r : r - qi * p.g;
      uint4 w[D / 32];
      float amax = 0.f, norm = 0.f;
      const uint16_t* src = static_cast<const uint16_t*>(p.q) + ((long long)(h * p.g + hd) * p.total_q + t.q0 + i0 + qi) * D + c * 16;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        w[k] = r < rows ? __ldg(reinterpret_cast<const uint4*>(src + (k >> 1) * 64) + (k & 1)) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float a = fabsf(__uint_as_float(u[j] << 16)), b = fabsf(__uint_as_float(u[j] & 0xffff0000u));
          amax = fmax3(amax, a, b);
          norm += a + b;
        }
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      norm += __shfl_xor_sync(0xffffffffu, norm, 1);
      norm += __shfl_xor_sync(0xffffffffu, norm, 2);
      const uint32_t e = __float_as_uint(amax) >> 23;              // biased exponent
      const uint32_t up = min(268u - e, 253u);                     // of the factor: largest |q| to [2^14, 2^15)
      const float inv = __uint_as_float(up << 23);
      unscale[i] = __uint_as_float((254u - up) << 23);
      // Infinite or NaN: scores that say nothing (all pages are then scored in 64 bits).
      if (!(norm <= kBig)) norm = INFINITY;
      if (c == 0 && r < rows && warp == 0) atomicMax(reinterpret_cast<int*>(norms + qi), __float_as_int(norm));   // >= 0
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t h2 = pack_f16x2(__uint_as_float(u[j] << 16) * inv, __uint_as_float(u[j] & 0xffff0000u) * inv);
          const int word = (k & 1) * 4 + j;
          qp[(k >> 1) * 4 + (word >> 1)][(word & 1) * 2 + i] = positive(h2);
          qm[(k >> 1) * 4 + (word >> 1)][(word & 1) * 2 + i] = negative(h2);
        }
      }
    }
    // ---- pages, 8 at a time: column rq of the products is page base + rq
    auto page_at = [&](int base) -> int {
      const int j = base + rq;
      if (j < begin || j >= end) return -1;
      const int pg = __ldg(table + j);
      if (pg < 0 || pg >= p.num_pages) {
        atomicExch(p.status, DEV_BAD_PAGE);
        return -1;
      }
      return pg;
    };
    int base = begin / 8 * 8 + warp * 8, pg = page_at(base);
    for (; base < end; base += kStepPages) {
      const int pg_now = pg;
      pg = page_at(base + kStepPages);
      uint4 lo[D / 64], hi[D / 64];
      float scale = 0.f;
#pragma unroll
      for (int k = 0; k < D / 64; ++k) lo[k] = hi[k] = make_uint4(0u, 0u, 0u, 0u);
      if (pg_now >= 0) {
        const long long ph = (long long)pg_now * p.Hkv + h;
        const uint8_t* row = p.bounds + ph * 2 * D + c * 16;
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          lo[k] = __ldg(reinterpret_cast<const uint4*>(row + k * 64));
          hi[k] = __ldg(reinterpret_cast<const uint4*>(row + D + k * 64));
        }
        scale = __ldg(p.k_scale + ph);
      }
      big = fmaxf(big, scale <= kBig ? scale : INFINITY);
      // Four sums of their own for the products that one takes in turn: a quarter of the rounding.
      float acc[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 64; ++k) {
        const uint32_t l[4] = {lo[k].x, lo[k].y, lo[k].z, lo[k].w}, u[4] = {hi[k].x, hi[k].y, hi[k].z, hi[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          mma_f16(acc[j], qp[k * 4 + j], e4m3x2_f16x2(u[j]), e4m3x2_f16x2_hi(u[j]));
          mma_f16(acc[j], qm[k * 4 + j], e4m3x2_f16x2(l[j]), e4m3x2_f16x2_hi(l[j]));
        }
      }
      const float s0 = __shfl_sync(0xffffffffu, scale, c * 8), s1 = __shfl_sync(0xffffffffu, scale, c * 8 + 4);
      __syncwarp();                          // the sums before have been read
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sums[warp][rq + 8 * i][2 * c] = ((acc[0][2 * i] + acc[1][2 * i]) + (acc[2][2 * i] + acc[3][2 * i])) * unscale[i] * s0;
        sums[warp][rq + 8 * i][2 * c + 1] = ((acc[0][2 * i + 1] + acc[1][2 * i + 1]) + (acc[2][2 * i + 1] + acc[3][2 * i + 1])) * unscale[i] * s1;
      }
      __syncwarp();
      // The largest of each query's heads; NaN wins.
      for (int x = lane; x < (i1 - i0) * 8; x += 32) {
        const int qi = x >> 3, j = base + (x & 7);
        if (j < begin || j >= end) continue;
        const int r0 = tiles > 1 ? 0 : qi * p.g, r1 = tiles > 1 ? heads : r0 + p.g;
        float* out = p.scores + ((long long)h * p.total_q + t.q0 + i0 + qi) * p.max_pages + j;
        float m = rt > 0 ? *out : -INFINITY;
        for (int r = r0; r < r1; ++r) {
          const float v = sums[warp][r][x & 7];
          m = v != v || v > m ? v : m;
        }
        *out = m;
      }
    }
  }
  // |error| of a score: products are exact, each of the 2 d / 64 products of 16 terms behind one another adds 17
  // numbers, off by 2^-23 of what they can come to at most, 448 scale |q|_1; four roundings more.
  big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));
  if (lane == 0) scale_max[warp] = big;
  __syncthreads();
  if (tid < i1 - i0) {
    for (int w = 1; w < kSelWarps; ++w) big = fmaxf(big, scale_max[w]);
    big = fmaxf(big, scale_max[0]);
    p.errors[((long long)h * p.total_q + t.q0 + i0 + tid) * p.chunks + chunk] =
        (2 * D / 64 * 17 + 4) * 1.1920929e-7f * 448.f * big * norms[tid];
  }
}

// Bits of a double, ordered as numbers: equal zeros, NaN above all.
__device__ __forceinline__ unsigned long long ordered(double x) {
  if (x != x) return ~0ull;
  const long long b = __double_as_longlong(x + 0.0);
  return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | (1ull << 63);
}

// Block: (query, K/V head).
template <int D>
__global__ void __launch_bounds__(kSelThreads) select_choose_kernel(const SelectParams p, const int in_smem) {
  extern __shared__ float local[];
  __shared__ int red[2][kSelWarps][2];
  __shared__ float redf[kSelWarps][3];
  constexpr int kFew = kSelThreads;          // pages near the border that are ranked in shared memory
  __shared__ unsigned long long few_keys[kFew];
  __shared__ int few_at[kFew];
  pdl_wait();                                // nothing of global memory before this
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % p.Hkv, q = blockIdx.x / p.Hkv;
  SelectParams one = p;
  one.qn = 1;
  Tile t;
  if (!find_tile(one, q, t)) return;
  const int seen = pages_seen(p, t, q - t.q0);
  const long long unit = (long long)h * p.total_q + q;
  int* out = p.out + unit * p.count;
  if (seen <= p.count) {
    for (int e = tid; e < p.count; e += kSelThreads) out[e] = e < seen ? e : -1;
    return;
  }
  for (int e = tid; e < p.first; e += kSelThreads) out[e] = e;
  for (int e = tid; e < p.last; e += kSelThreads) out[p.count - p.last + e] = seen - p.last + e;
  const int n = seen - p.first - p.last, k = p.count - p.first - p.last;   // k of n candidates
  if (k == 0) return;
  float* scores = p.scores + unit * p.max_pages + p.first;
  float* v = in_smem ? local : scores;
  // ---- candidates and their range; NaN ranks above all
  float low = INFINITY, high = -INFINITY, eps = 0.f;
  bool strange = false;
  for (int i = tid; i < n; i += kSelThreads) {
    float x = scores[i];
    if (x != x) x = INFINITY;
    else {
      strange |= !(fabsf(x) <= kBig);
      low = fminf(low, x);
      high = fmaxf(high, x);
    }
    v[i] = x;
  }
  for (int i = p.first / p.chunk + tid; i <= (seen - p.last - 1) / p.chunk; i += kSelThreads)
    eps = fmaxf(eps, p.errors[unit * p.chunks + i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
    high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
    eps = fmaxf(eps, __shfl_xor_sync(0xffffffffu, eps, o));
  }
  if (lane == 0) {
    redf[warp][0] = low;
    redf[warp][1] = high;
    redf[warp][2] = eps;
  }
  strange = __syncthreads_or(strange) != 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) {
    low = fminf(low, redf[w][0]);
    high = fmaxf(high, redf[w][1]);
    eps = fmaxf(eps, redf[w][2]);
  }
  // Sums over all threads of two small counts; every second call has its own slots.
  int turn = 0;
  auto count2 = [&](int a, int b) -> int2 {
    a = __reduce_add_sync(0xffffffffu, a);
    b = __reduce_add_sync(0xffffffffu, b);
    if (lane == 0) {
      red[turn][warp][0] = a;
      red[turn][warp][1] = b;
    }
    __syncthreads();
    a = b = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
      a += red[turn][w][0];
      b += red[turn][w][1];
    }
    turn ^= 1;
    return make_int2(a, b);
  };
  auto above = [&](float x) -> int {
    int m = 0;
    for (int i = tid; i < n; i += kSelThreads) m += v[i] > x ? 1 : 0;
    return count2(m, 0).x;
  };
  // ---- the border: pages above `top` are among the k best for sure, those below `bottom` are not
  float top, bottom;
  const bool all = strange || !(eps <= kBig / 131072.f);           // scores that may have overflowed: none is sure
  if (all) {
    top = INFINITY;
    bottom = -INFINITY;
  } else if (above(kBig) >= k) {             // enough NaN pages to fill the list
    top = INFINITY;
    bottom = kBig;
  } else {
    // The k-th largest of the scores lies in [low, high]: at least k are >= low, fewer than k above high.
    for (int it = 0; it < 64 && high - low > eps; ++it) {
      const float mid = low + (high - low) * 0.5f;
      if (mid <= low || mid >= high) break;
      if (above(mid) < k) high = mid;
      else low = mid;
    }
    top = high + 2.01f * eps;
    bottom = low - 2.01f * eps;
  }
  int in = 0, near = 0;
  for (int i = tid; i < n; i += kSelThreads) {
    const float x = v[i];
    if (x > top) ++in;
    else if (x >= bottom) ++near;
  }
  const int2 both = count2(in, near);
  const int need = k - both.x, m = both.y;   // of the m pages near the border
  const float emit = m == need ? (all ? -INFINITY : nextafterf(bottom, -INFINITY)) : fminf(top, kBig);
  if (m != need) {
    // ---- these in 64 bits, in the order of their numbers
    unsigned long long* keys = m <= kFew ? few_keys : p.exact + unit * p.max_pages;
    int* at = m <= kFew ? few_at : p.near + unit * p.max_pages;
    for (int i0 = 0, found = 0; i0 < n; i0 += kSelThreads) {
      const int i = i0 + tid;
      const float x = i < n ? v[i] : 0.f;
      const bool is = i < n && !(x > top) && x >= bottom;
      const uint32_t votes = __ballot_sync(0xffffffffu, is);
      if (lane == 0) red[turn][warp][0] = __popc(votes);
      __syncthreads();
      int before = found;
#pragma unroll
      for (int w = 0; w < kSelWarps; ++w) {
        if (w < warp) before += red[turn][w][0];
        found += red[turn][w][0];
      }
      turn ^= 1;
      if (is) at[before + __popc(votes & ((1u << lane) - 1))] = i;
    }
    __syncthreads();
    const int* table = p.table + (long long)t.b * p.max_pages;
    for (int a = warp; a < m; a += kSelWarps) {
      const int pg = __ldg(table + p.first + at[a]);
      double best = -INFINITY;
      if (eps == 0.f) best = 0.0;            // every scale is 0, or q
      else if (pg >= 0 && pg < p.num_pages) {
        constexpr int COLS = D / 32;
        const long long ph = (long long)pg * p.Hkv + h;
        const uint8_t* row = p.bounds + ph * 2 * D + lane * COLS;
        float lo[4], hi[4];
        if constexpr (COLS == 4) {
          e4m3x4_to_f32(__ldg(reinterpret_cast<const uint32_t*>(row)), lo[0], lo[1], lo[2], lo[3]);
          e4m3x4_to_f32(__ldg(reinterpret_cast<const uint32_t*>(row + D)), hi[0], hi[1], hi[2], hi[3]);
        } else {
          e4m3x4_to_f32(__ldg(reinterpret_cast<const uint16_t*>(row)), lo[0], lo[1], lo[2], lo[3]);
          e4m3x4_to_f32(__ldg(reinterpret_cast<const uint16_t*>(row + D)), hi[0], hi[1], hi[2], hi[3]);
        }
        const double scale = (double)__ldg(p.k_scale + ph);
        bool nan = false;
        for (int r = 0; r < p.g; ++r) {
          const uint16_t* src = static_cast<const uint16_t*>(p.q) + ((long long)(h * p.g + r) * p.total_q + q) * D + lane * COLS;
          double s = 0.0;
#pragma unroll
          for (int x = 0; x < COLS; ++x) {
            const float y = __uint_as_float((uint32_t)__ldg(src + x) << 16);
            const float plus = y > 0.f || y != y ? y : 0.f, minus = y < 0.f || y != y ? y : 0.f;
            s = fma((double)plus, (double)hi[x], s);
            s = fma((double)minus, (double)lo[x], s);
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          nan |= s != s;
          best = fmax(best, s);
        }
        best = nan ? __longlong_as_double(0x7ff8000000000000ll) : best * scale;
      }
      if (lane == 0) keys[a] = ordered(best);
    }
    __syncthreads();
    if (m <= kFew) {
      if (tid < m) {                         // rank: better ones, and equal ones before it
        const unsigned long long mine = keys[tid];
        int ahead = 0;
        for (int a = 0; a < m; ++a) ahead += keys[a] > mine || (keys[a] == mine && a < tid) ? 1 : 0;
        v[at[tid]] = ahead < need ? INFINITY : -INFINITY;
      }
    } else {
      // The need-th largest key, bit by bit; then of the keys equal to it the first ones.
      unsigned long long key = 0;
      for (int bit = 63; bit >= 0; --bit) {
        const unsigned long long trial = key | (1ull << bit);
        int enough = 0;
        for (int a = tid; a < m; a += kSelThreads) enough += keys[a] >= trial ? 1 : 0;
        if (count2(enough, 0).x >= need) key = trial;
      }
      int better = 0;
      for (int a = tid; a < m; a += kSelThreads) better += keys[a] > key ? 1 : 0;
      const int equal_need = need - count2(better, 0).x;
      for (int a0 = 0, found = 0; a0 < m; a0 += kSelThreads) {
        const int a = a0 + tid;
        const bool equal = a < m && keys[a] == key;
        const uint32_t votes = __ballot_sync(0xffffffffu, equal);
        if (lane == 0) red[turn][warp][0] = __popc(votes);
        __syncthreads();
        int before = found;
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w) {
          if (w < warp) before += red[turn][w][0];
          found += red[turn][w][0];
        }
        turn ^= 1;
        const bool take = a < m && (keys[a] > key || (equal && before + __popc(votes & ((1u << lane) - 1)) < equal_need));
        if (a < m) v[at[a]] = take ? INFINITY : -INFINITY;
      }
    }
    __syncthreads();
  }
  // ---- out, ascending
  for (int i0 = 0, found = 0; i0 < n; i0 += kSelThreads) {
    const int i = i0 + tid;
    const bool is = i < n && v[i] > emit;
    const uint32_t votes = __ballot_sync(0xffffffffu, is);
    if (lane == 0) red[turn][warp][0] = __popc(votes);
    __syncthreads();
    int before = found;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
      if (w < warp) before += red[turn][w][0];
      found += red[turn][w][0];
    }
    turn ^= 1;
    const int place = before + __popc(votes & ((1u << lane) - 1));
    if (is && place < k) out[p.first + place] = p.first + i;
  }
}

// Pages of a chunk: as many as leave 8 CTAs per SM, from one step of a CTA on.
int chunk_pages(long long units, int max_pages, int sms) {
  int steps = 8;
  while (steps > 1 && units * ((max_pages + steps * kStepPages - 1) / (steps * kStepPages)) < 8LL * sms) steps /= 2;
  return steps * kStepPages;
}

}  // namespace

// [Hkv][total_q] rows: scores, the 64-bit keys and numbers of pages near the border, the chunks' errors.
SelectWs select_ws(int Hkv, int total_q, int max_pages) {
  const auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  const size_t rows = (size_t)Hkv * total_q, chunks = ((size_t)max_pages + kStepPages - 1) / kStepPages;
  SelectWs w;
  w.exact = up(rows * max_pages * 4);
  w.near = w.exact + up(rows * max_pages * 8);
  w.errors = w.near + up(rows * max_pages * 4);
  w.total = w.errors + up(rows * chunks * 4);
  return w;
}

cudaError_t launch_select_pages(SelectParams p, int d, int sms, cudaStream_t s) {
  p.page_shift = p.page == 16 ? 4 : p.page == 32 ? 5 : p.page == 64 ? 6 : 7;
  // Queries of a tile: as many as fill 16 rows, but no more than a sequence has.
  p.qn = p.g >= 16 ? 1 : (p.max_q < 16 / p.g ? p.max_q : 16 / p.g);
  const long long slots = p.qn > 1 ? (long long)p.total_q / p.qn + p.B : p.total_q, units = slots * p.Hkv;
  p.chunk = chunk_pages(units, p.max_pages, sms);
  p.chunks = (p.max_pages + p.chunk - 1) / p.chunk;
  const long long grid = units * p.chunks, lists = (long long)p.total_q * p.Hkv;
  if (slots > 0x7fffffffLL || grid > 0x7fffffffLL || lists > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  if (p.max_pages > p.count)                 // (else every list holds all pages)
    e = d == 64 ? launch_pdl(select_score_kernel<64>, dim3((unsigned)grid), dim3(kSelThreads), 0, s, p)
                : launch_pdl(select_score_kernel<128>, dim3((unsigned)grid), dim3(kSelThreads), 0, s, p);
  if (e != cudaSuccess) return e;
  const size_t bytes = (size_t)p.max_pages * 4;
  const int in_smem = bytes <= 40 * 1024 ? 1 : 0;      // (longer tables: in the workspace)
  return d == 64 ? launch_pdl(select_choose_kernel<64>, dim3((unsigned)lists), dim3(kSelThreads), in_smem ? bytes : 0, s, p, in_smem)
                 : launch_pdl(select_choose_kernel<128>, dim3((unsigned)lists), dim3(kSelThreads), in_smem ? bytes : 0, s, p, in_smem);
}

}  // namespace attn
