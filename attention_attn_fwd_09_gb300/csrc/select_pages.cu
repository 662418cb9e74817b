// The pages of a paged e4m3 cache that each query is to read, by an upper bound of its scores there.
//
// A page's bounds hold its smallest and largest code per column (lo, hi).  No key of the page can
// score more against q than
//     s(q, page) = scale_page sum_c max(q_c, 0) hi_c + min(q_c, 0) lo_c,
// and the heads of a group, which share a list, go by the largest of theirs.  The first pages (which
// much attention falls on whatever the query) and the last ones (the nearest keys) are always
// listed, the best of the others fill the list, ascending; a sequence with few enough pages lists all.
//
// What is chosen is what scores in 64-bit floating point choose, each head's sum rounded once (equal ones go by
// number), whatever order a sum is taken in: the kernels score in fp32 with a bound on their error, and only pages
// too near the border to tell are scored again, by exact sums.  So the list depends on nothing but the query and
// the bounds.
//
// Two dependent launches:
//   * scores, bound by the bounds' bytes (2 d per page and K/V head): a warp takes 16 pages as the rows
//     of mma.m16n8k16 (read straight into the fragments: a lane's share of a page is 16 neighbouring
//     columns), the columns are queries x heads of a group, 8 or 16 of them; the products run over
//     [max(q, 0), min(q, 0)] against [hi, lo].  f16 holds the codes and, scaled by a power of two per row, q
//     (exact down to 2^-31 of the row's largest component, off by 2^-39 of it below).  The work is cut
//     evenly: all units' steps of 16 pages end to end, every warp an equal run.  64 ragged sequences of up
//     to 32768 keys in pages of 32: 22.5 us profiled with cold caches, 3.1 TB/s (37 us with pages as the
//     columns of the same instruction, which takes twice the products);
//   * choice, bound by latency: a CTA per query and K/V head looks for the border with histograms
//     (14.6 us there; bisection took 15 steps of 600 cycles).
// Both in a graph: those sequences 28 us, one sequence of 32768 keys 12, 8 x 4 drafted tokens of 32 heads on one 20.
#include <cstdint>
#include <mutex>

#include "cache.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kScoreThreads = 128, kScoreWarps = kScoreThreads / 32, kScoreCtas = 4;   // CTAs per SM
constexpr int kStep = 16;                    // pages that a warp scores at once
constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;
constexpr float kBig = 3.0e38f, kTiny = 1.17549435e-38f;          // 2^-126

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t positive(uint32_t x) {
  const __half2 z = __float2half2_rn(0.f), r = __hmax2(*reinterpret_cast<const __half2*>(&x), z);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t negative(uint32_t x) {
  const __half2 z = __float2half2_rn(0.f), r = __hmin2(*reinterpret_cast<const __half2*>(&x), z);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float max_nan(float a, float b) {       // NaN wins
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A sequence's queries and keys.
struct Seq {
  int q0, n, len;
  __device__ __forceinline__ Seq(const SelectParams& p, int b) {
    q0 = __ldg(p.cu_q + b);
    n = __ldg(p.cu_q + b + 1) - q0;
    len = __ldg(p.kv_lens + b);
  }
  __device__ __forceinline__ bool wrong(const SelectParams& p, int b) const {
    const int c1 = q0 + n;
    return q0 < 0 || n < 0 || c1 < 0 || n > p.max_q || len < 0 || len > p.max_len || (p.causal && n > len) ||
           (b == 0 && q0 != 0) || (b == p.B - 1 && c1 != p.total_q);
  }
  // Pages that query i sees.
  __device__ __forceinline__ int seen(const SelectParams& p, int i) const {
    const int keys = p.causal ? len - n + i + 1 : len;
    return (keys + p.page - 1) >> p.page_shift;
  }
  // Steps of 16 pages (numbers 16 s .. 16 s + 15) that hold candidates of its last query: [first_step, first_step + steps).
  __device__ __forceinline__ int steps(const SelectParams& p) const {
    const int all = seen(p, n - 1), end = all - p.last;
    return n == 0 || all <= p.count || end <= p.first ? 0 : (end + kStep - 1) / kStep - p.first / kStep;
  }
  __device__ __forceinline__ int tiles(const SelectParams& p) const { return (n + p.qn - 1) / p.qn; }
};

// Scores [K/V head][query][max_pages] and, per step of 16 pages, a bound on their error.  A unit is a tile of
// queries of one sequence (as many as make 8 NT rows with their heads) and a K/V head.
template <int D, int NT>
__global__ void __launch_bounds__(kScoreThreads, kScoreCtas) select_score_kernel(const SelectParams p) {
  constexpr int KS = D / 16;                 // products of 16 columns
  __shared__ float rows_of[kScoreWarps][kStep][8 * NT + 1];        // groups of other sizes than powers of two
  __shared__ float row_norm[kScoreWarps][8 * NT];
  __shared__ long long starts[kScoreThreads], sums[kScoreWarps];
  pdl_wait();                                // nothing of global memory before this
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = lane & 3, rq = lane >> 2;
  // ---- the run of steps of this warp; thread t adds up sequences [t per_thread, ...)
  const int per_thread = (p.B + kScoreThreads - 1) / kScoreThreads;
  const int b_lo = min(tid * per_thread, p.B), b_hi = min(b_lo + per_thread, p.B);
  long long mine = 0;
  bool wrong = false;
  for (int b = b_lo; b < b_hi; ++b) {
    const Seq s(p, b);
    const bool w = s.wrong(p, b);
    wrong |= w;
    if (!w) mine += (long long)s.tiles(p) * s.steps(p);
  }
  mine *= p.Hkv;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sums[warp] = incl;
  const bool bad = __syncthreads_or(wrong) != 0;
  if (bad) {
    if (tid == 0) atomicExch(p.status, DEV_BAD_OFFSETS);
    return;
  }
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kScoreWarps; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  starts[tid] = before;
  __syncthreads();
  const long long warps = (long long)gridDim.x * kScoreWarps, run = (total + warps - 1) / warps;
  // (neighbouring runs on different SMs: few units leave no SM with several)
  const long long rs = run * ((long long)warp * gridDim.x + blockIdx.x), re = min(rs + run, total);
  if (rs >= total) return;
  int at = 0;                                // the last thread whose sequences start at or before rs
#pragma unroll
  for (int i = 0; i < kScoreThreads / 32; ++i) at += __popc(__ballot_sync(0xffffffffu, starts[i * 32 + lane] <= rs));
  int b = (at - 1) * per_thread;
  long long f = starts[at - 1];              // first step of sequence b
  Seq seq(p, b);
  int steps = seq.steps(p);
  long long all = (long long)seq.tiles(p) * p.Hkv * steps;
  while (f + all <= rs) {
    f += all;
    seq = Seq(p, ++b);
    steps = seq.steps(p);
    all = (long long)seq.tiles(p) * p.Hkv * steps;
  }
  int unit = (int)((rs - f) / steps), step = (int)((rs - f) - (long long)unit * steps);
  constexpr int ROWS = 8 * NT;
  const int row_tiles = p.g > ROWS ? (p.g + ROWS - 1) / ROWS : 1;  // of 16 heads, when a group has more
  const bool pow2 = (p.g & (p.g - 1)) == 0;

  for (long long left = re - rs; left > 0;) {
    const int tile = unit / p.Hkv, h = unit - tile * p.Hkv, i0 = tile * p.qn, nq = min(p.qn, seq.n - i0);
    const int todo = (int)min((long long)(steps - step), left);    // steps of this unit here
    const int begin = p.first, end = seq.seen(p, i0 + nq - 1) - p.last;      // candidates of the tile's queries
    const int* table = p.table + (long long)b * p.max_pages;
    const long long out_row = (long long)h * p.total_q + seq.q0 + i0;        // of the first query
    auto page_at = [&](int j) -> int {
      if (j < begin || j >= end) return -1;
      const int pg = __ldg(table + j);
      if (pg < 0 || pg >= p.num_pages) {
        atomicExch(p.status, DEV_BAD_PAGE);
        return -1;
      }
      return pg;
    };
    for (int rt = 0; rt < row_tiles; ++rt) {
      int j = (p.first / kStep + step) * kStep + rq;               // this lane's pages: j and j + 8
      int pg[2] = {page_at(j), page_at(j + 8)};
      const int heads = min(p.g - rt * ROWS, ROWS), rows = row_tiles > 1 ? heads : nq * p.g;
      // ---- Q: row r is query r / g, head r % g; this lane's columns of rows rq (and rq + 8)
      uint32_t qp[NT][KS][2], qm[NT][KS][2];
      float us[NT][2];                       // what undoes the scaling of rows 2 c, 2 c + 1
      __syncwarp();                          // the norms before have been read
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int r = rq + 8 * i, qi = row_tiles > 1 ? 0 : r / p.g, hd = row_tiles > 1 ? rt * ROWS + r : r - qi * p.g;
        uint4 w[D / 32];
        float amax = 0.f, sum = 0.f;
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + ((long long)(h * p.g + hd) * p.total_q + seq.q0 + i0 + qi) * D + c * 16;
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
          w[k] = r < rows ? __ldg(reinterpret_cast<const uint4*>(src + (k >> 1) * 64) + (k & 1)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float y = fabsf(__uint_as_float(u[x] << 16)), z = fabsf(__uint_as_float(u[x] & 0xffff0000u));
            amax = fmax3(amax, y, z);
            sum += y + z;
          }
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const uint32_t e = __float_as_uint(amax) >> 23;            // biased exponent
        const uint32_t up = min(268u - e, 253u);                   // of the factor: largest |q| to [2^14, 2^15)
        const float inv = __uint_as_float(up << 23), unscale = __uint_as_float((254u - up) << 23);
        us[i][0] = __shfl_sync(0xffffffffu, unscale, c * 8);
        us[i][1] = __shfl_sync(0xffffffffu, unscale, c * 8 + 4);
        // Infinite or NaN: scores that say nothing (all pages are then scored exactly).
        if (c == 0) row_norm[warp][r] = r < rows ? (sum <= kBig ? sum : INFINITY) : 0.f;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t h2 = pack_f16x2(__uint_as_float(u[x] << 16) * inv, __uint_as_float(u[x] & 0xffff0000u) * inv);
            const int word = (k & 1) * 4 + x;
            qp[i][(k >> 1) * 4 + (word >> 1)][word & 1] = positive(h2);
            qm[i][(k >> 1) * 4 + (word >> 1)][word & 1] = negative(h2);
          }
        }
      }
      __syncwarp();
      float norm = 0.f;                      // lane qi: the largest |q|_1 of query qi's heads here
      if (lane < nq) {
        const int r0 = row_tiles > 1 ? 0 : lane * p.g, r1 = row_tiles > 1 ? heads : r0 + p.g;
        for (int r = r0; r < r1; ++r) norm = fmaxf(norm, row_norm[warp][r]);
      }
      // |error| of a score: products are exact, and each of the 2 d / 64 products of 16 terms behind one another
      // adds 17 numbers, off by 2^-23 of what they can come to at most, 448 scale |q|_1; four roundings more.
      norm *= (2 * D / 64 * 17 + 4) * 1.1920929e-7f * 448.f;

      for (int s = 0; s < todo; ++s, j += kStep) {
        float scale[2];
        uint4 lo[2][D / 64], hi[2][D / 64];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const long long ph = (long long)max(pg[x], 0) * p.Hkv + h;
          const uint8_t* row = p.bounds + ph * 2 * D + c * 16;     // (no page: page 0, which counts for nothing)
#pragma unroll
          for (int k = 0; k < D / 64; ++k) {
            lo[x][k] = __ldg(reinterpret_cast<const uint4*>(row + k * 64));
            hi[x][k] = __ldg(reinterpret_cast<const uint4*>(row + D + k * 64));
          }
          scale[x] = __ldg(p.k_scale + ph);
        }
        const bool got[2] = {pg[0] >= 0, pg[1] >= 0};
        if (s + 1 < todo) {
          pg[0] = page_at(j + kStep);
          pg[1] = page_at(j + kStep + 8);
        }
        // Four sums of their own for the products that one takes in turn: a quarter of the rounding.
        float acc[NT][4][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[i][x][0] = acc[i][x][1] = acc[i][x][2] = acc[i][x][3] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          const uint32_t l0[4] = {lo[0][k].x, lo[0][k].y, lo[0][k].z, lo[0][k].w}, l1[4] = {lo[1][k].x, lo[1][k].y, lo[1][k].z, lo[1][k].w};
          const uint32_t u0[4] = {hi[0][k].x, hi[0][k].y, hi[0][k].z, hi[0][k].w}, u1[4] = {hi[1][k].x, hi[1][k].y, hi[1][k].z, hi[1][k].w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t a0 = e4m3x2_f16x2(u0[x]), a1 = e4m3x2_f16x2(u1[x]), a2 = e4m3x2_f16x2_hi(u0[x]), a3 = e4m3x2_f16x2_hi(u1[x]);
            const uint32_t d0 = e4m3x2_f16x2(l0[x]), d1 = e4m3x2_f16x2(l1[x]), d2 = e4m3x2_f16x2_hi(l0[x]), d3 = e4m3x2_f16x2_hi(l1[x]);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              mma_f16(acc[i][x], a0, a1, a2, a3, qp[i][k * 4 + x][0], qp[i][k * 4 + x][1]);
              mma_f16(acc[i][x], d0, d1, d2, d3, qm[i][k * 4 + x][0], qm[i][k * 4 + x][1]);
            }
          }
        }
        float v[NT][2][2];                   // rows 2 c, 2 c + 1 (+ 8 i), pages j, j + 8
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y)
              v[i][y][x] = ((acc[i][0][2 * x + y] + acc[i][1][2 * x + y]) + (acc[i][2][2 * x + y] + acc[i][3][2 * x + y])) * us[i][y] * scale[x];
        auto put = [&](int qi, int x, float y) {         // the largest over all row tiles so far
          if (!got[x]) return;
          float* out = p.scores + (out_row + qi) * p.max_pages + j + 8 * x;
          *out = rt > 0 ? max_nan(*out, y) : y;
        };
        if (pow2) {                          // the largest of each query's heads, lane to lane
          if (p.g == 1) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int qi = 8 * i + 2 * c + y;
                if (qi >= nq) continue;
                put(qi, 0, v[i][y][0]);
                put(qi, 1, v[i][y][1]);
              }
          } else {
            float m[NT][2];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                float y = max_nan(v[i][0][x], v[i][1][x]);
                if (p.g >= 4) y = max_nan(y, __shfl_xor_sync(0xffffffffu, y, 1));
                if (p.g >= 8) y = max_nan(y, __shfl_xor_sync(0xffffffffu, y, 2));
                m[i][x] = y;
              }
            if (NT > 1 && p.g >= 16) {
              m[0][0] = max_nan(m[0][0], m[NT - 1][0]);
              m[0][1] = max_nan(m[0][1], m[NT - 1][1]);
            }
            if ((2 * c & (min(p.g, 8) - 1)) == 0) {
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                const int qi = row_tiles > 1 ? 0 : (8 * i + 2 * c) / p.g;
                if (qi >= nq || (i > 0 && p.g >= 16)) continue;
                put(qi, 0, m[i][0]);
                put(qi, 1, m[i][1]);
              }
            }
          }
        } else {
          __syncwarp();                      // the rows before have been read
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int y = 0; y < 2; ++y) rows_of[warp][rq + 8 * x][8 * i + 2 * c + y] = v[i][y][x];
          __syncwarp();
          for (int z = lane; z < nq * kStep; z += 32) {
            const int qi = z / kStep, x = z % kStep, page = j - rq + x;
            const int r0 = row_tiles > 1 ? 0 : qi * p.g, r1 = row_tiles > 1 ? heads : r0 + p.g;
            float m = rows_of[warp][x][r0];
            for (int r = r0 + 1; r < r1; ++r) m = max_nan(m, rows_of[warp][x][r]);
            if (page < begin || page >= end) continue;
            float* out = p.scores + (out_row + qi) * p.max_pages + page;
            *out = rt > 0 ? max_nan(*out, m) : m;
          }
        }
        const float s0 = got[0] ? (scale[0] <= kBig ? scale[0] : INFINITY) : 0.f, s1 = got[1] ? (scale[1] <= kBig ? scale[1] : INFINITY) : 0.f;
        const float top_scale = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(s0, s1))));
        // 0 only where q or the scales are: what underflows here or in a score stays below the smallest normal number.
        const float error = norm > 0.f && top_scale > 0.f ? fmaxf(norm * top_scale, kTiny) : 0.f;
        if (lane < nq) {
          float* out = p.errors + (out_row + lane) * p.groups + p.first / kStep + step + s;
          *out = rt > 0 ? fmaxf(*out, error) : error;
        }
      }
    }
    left -= todo;
    step += todo;
    if (left > 0 && step == steps) {         // the next unit, or the next sequence that has any
      step = 0;
      if (++unit == seq.tiles(p) * p.Hkv) {
        unit = 0;
        do {
          seq = Seq(p, ++b);
          steps = seq.steps(p);
        } while (steps == 0);
      }
    }
  }
}

// Bits of a double, ordered as numbers: equal zeros, NaN above all.
__device__ __forceinline__ unsigned long long ordered(double x) {
  if (x != x) return ~0ull;
  const long long b = __double_as_longlong(x + 0.0);
  return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | (1ull << 63);
}
// The same of a float, as a signed number.
__device__ __forceinline__ int ordered32(float x) {
  const int b = __float_as_int(x);
  return b < 0 ? b ^ 0x7fffffff : b;
}
__device__ __forceinline__ float unordered32(int b) { return __int_as_float(b < 0 ? b ^ 0x7fffffff : b); }

// The sum over a warp of products m n 2^(s - 142) (signed; m n below 2^12, s up to 267) that lie too far apart for
// 64 bits, rounded once: nine digits of 32 bits, each added up by itself (128 products stay below 2^50).  A lane
// brings up to four, as 512 m n + s.
__device__ __noinline__ double far_sum(int4 terms) {
  constexpr int DIGITS = 9;
  const int t[4] = {terms.x, terms.y, terms.z, terms.w};
  uint32_t digit[DIGITS];
  long long carry = 0;
#pragma unroll
  for (int i = 0; i < DIGITS; ++i) {
    long long sum = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if ((t[x] >> 5 & 15) == i) sum += (long long)(t[x] >> 9) * (1ll << (t[x] & 31));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    sum += carry;
    digit[i] = (uint32_t)sum;
    carry = sum >> 32;                       // (rounds down)
  }
  const bool negative = carry < 0;           // the sum is below 2^288: 0 or -1
  if (negative) {
    uint32_t one = 1;
#pragma unroll
    for (int i = 0; i < DIGITS; ++i) {
      digit[i] = ~digit[i] + one;
      one = one != 0 && digit[i] == 0 ? 1 : 0;
    }
  }
  // The leading 64 bits, the last of them set if any behind is: the conversion then rounds as the whole sum would.
  uint32_t a = 0, b = 0, c = 0, rest = 0;
  int top = 0;
#pragma unroll
  for (int i = DIGITS - 1; i >= 0; --i) {
    if (a == 0) {
      a = digit[i];
      b = i > 0 ? digit[i > 0 ? i - 1 : 0] : 0u;
      c = i > 1 ? digit[i > 1 ? i - 2 : 0] : 0u;
      rest = 0;
      top = i;
    } else if (i < top - 2) {
      rest |= digit[i];
    }
  }
  if (a == 0) return 0.0;
  const int z = __clz(a);
  const unsigned long long lead = (((unsigned long long)a << 32 | b) << z) | (z > 0 ? c >> (32 - z) : 0u);
  const double x = __ull2double_rn(lead | ((c << z | rest) != 0 ? 1u : 0u)) *
                   __longlong_as_double((long long)(32 * (top - 1) - z - 142 + 1023) << 52);
  return negative ? -x : x;
}

// The exact score of page pg for packed query q and heads r0 .. r0 + 3 of the group of K/V head h, as ordered()
// bits: each head's sum rounded once to 64-bit floating point, times the scale; by a warp.  Codes are m 2^x with 4
// bits of m and q's components with 8, so that their products, as whole numbers times one power of two, add up
// exactly in 64 bits where q's components lie within 2^29 of each other, elsewhere in more (far_sum).  Sums with
// infinities and NaN, where no rounding counts, are taken in doubles (all by doubles, two pages took 11000 cycles).
constexpr int kExactHeads = 4;
template <int D>
__device__ unsigned long long exact_score(const SelectParams& p, int q, int h, int r0, int pg) {
  constexpr int COLS = D / 32;
  const int lane = threadIdx.x & 31;
  uint32_t w[kExactHeads][2];
#pragma unroll
  for (int r = 0; r < kExactHeads; ++r) {
    const uint16_t* src = static_cast<const uint16_t*>(p.q) + ((long long)(h * p.g + min(r0 + r, p.g - 1)) * p.total_q + q) * D + lane * COLS;
    if constexpr (COLS == 4) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(src));
      w[r][0] = u.x;
      w[r][1] = u.y;
    } else {
      w[r][0] = __ldg(reinterpret_cast<const uint32_t*>(src));
    }
  }
  const long long ph = (long long)pg * p.Hkv + h;
  const uint8_t* row = p.bounds + ph * 2 * D + lane * COLS;
  const uint32_t lo = COLS == 4 ? __ldg(reinterpret_cast<const uint32_t*>(row)) : __ldg(reinterpret_cast<const uint16_t*>(row));
  const uint32_t hi = COLS == 4 ? __ldg(reinterpret_cast<const uint32_t*>(row + D)) : __ldg(reinterpret_cast<const uint16_t*>(row + D));
  const float scale = __ldg(p.k_scale + ph);
  bool nan = false;
#pragma unroll
  for (int x = 0; x < COLS; ++x) nan |= (lo >> 8 * x & 0x7f) == 0x7f || (hi >> 8 * x & 0x7f) == 0x7f;
  if (__any_sync(0xffffffffu, nan)) return ~0ull;
  double own = -INFINITY;                    // of head r0 + lane
#pragma unroll
  for (int r = 0; r < kExactHeads; ++r) {    // (behind the last head: the last again)
    int top = 1;
#pragma unroll
    for (int x = 0; x < COLS; ++x) top = max(top, (int)(w[r][x >> 1] >> (x & 1) * 16 + 7 & 0xff));
    top = (int)__reduce_max_sync(0xffffffffu, (unsigned)top);
    const bool strange = top == 255;         // an infinity or NaN
    bool far = false;
    long long sum = 0;
    int terms[4] = {0, 0, 0, 0};             // for far_sum
#pragma unroll
    for (int x = 0; x < COLS; ++x) {
      const uint32_t y = w[r][x >> 1] >> (x & 1) * 16 & 0xffffu, e = y >> 7 & 0xff;
      const int m = (int)((y & 0x7f) | (e ? 0x80 : 0)), below = top - max((int)e, 1);
      far |= m != 0 && below > 29;
      const uint32_t code = ((y >> 15 ? lo : hi) >> 8 * x) & 0xff, ce = code >> 3 & 15;
      const int n = (int)((code & 7) | (ce ? 8 : 0));
      const int product = (y >> 15) != (code >> 7) ? -m * n : m * n;
      terms[x] = product * 512 + max((int)e, 1) - 1 + max((int)ce, 1) - 1;
      sum += (long long)product * (1ll << (max(29 - below, 0) + max((int)ce, 1) - 1));
    }
    double s;
    if (!strange && __any_sync(0xffffffffu, far)) {
      s = far_sum(make_int4(terms[0], terms[1], terms[2], terms[3]));
    } else if (!strange) {
      const unsigned a = __reduce_add_sync(0xffffffffu, (unsigned)sum & 0xffffffu);
      const unsigned b = __reduce_add_sync(0xffffffffu, (unsigned)(sum >> 24) & 0xffffffu);
      const int d = __reduce_add_sync(0xffffffffu, (int)(sum >> 48));
      s = (double)((long long)a + ((long long)b << 24) + ((long long)d << 48)) * __longlong_as_double((long long)(top - 172 + 1023) << 52);
    } else {
      s = 0.0;
#pragma unroll
      for (int x = 0; x < COLS; ++x) {
        const float y = __uint_as_float((w[r][x >> 1] >> (x & 1) * 16) << 16);
        const float plus = y > 0.f || y != y ? y : 0.f, minus = y < 0.f || y != y ? y : 0.f;
        float l, u, unused;
        e4m3x4_to_f32(lo >> 8 * x & 0xff, l, unused, unused, unused);
        e4m3x4_to_f32(hi >> 8 * x & 0xff, u, unused, unused, unused);
        s = fma((double)plus, (double)u, s);
        s = fma((double)minus, (double)l, s);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    }
    if (lane == r) own = s;
  }
  const unsigned long long key = lane < kExactHeads ? ordered(own * (double)scale) : 0ull;
  const unsigned high = __reduce_max_sync(0xffffffffu, (unsigned)(key >> 32));
  const unsigned low = __reduce_max_sync(0xffffffffu, (unsigned)(key >> 32) == high ? (unsigned)key : 0u);
  return (unsigned long long)high << 32 | low;
}

// Block: (query, K/V head).
template <int D>
__global__ void __launch_bounds__(kSelThreads) select_choose_kernel(const SelectParams p, const int in_smem) {
  extern __shared__ float local[];
  constexpr int kBins = 256, kFew = kSelThreads;         // kFew: pages near the border that are ranked in shared memory
  __shared__ __align__(16) int bins[2][kBins + 4];       // [kBins]: above the range
  __shared__ int red[2][kSelWarps][2];
  __shared__ int4 redf[kSelWarps];
  __shared__ unsigned long long few_keys[kFew];
  __shared__ int few_at[kFew];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  bins[0][tid] = bins[1][tid] = 0;
  if (tid == 0) bins[0][kBins] = bins[1][kBins] = 0;
  pdl_wait();                                // nothing of global memory before this
  pdl_trigger();
  const int h = blockIdx.x % p.Hkv, q = blockIdx.x / p.Hkv;
  const long long unit = (long long)h * p.total_q + q;
  float* scores = p.scores + unit * p.max_pages;
  // The first scores on their way already; what they say of pages that are no candidates is not looked at.
  constexpr int kAhead = 4;
  float ahead[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) ahead[i] = p.first + i * kSelThreads + tid < p.max_pages ? scores[p.first + i * kSelThreads + tid] : 0.f;
  // ---- the query's sequence, the last that starts at or before it
  int b = -1;
  {
    bool wrong = false;
    auto look = [&](int i) -> bool {
      const Seq s(p, i);
      wrong |= s.wrong(p, i);
      return s.q0 <= q;
    };
    if (p.B <= kSelThreads) {
      const bool below = tid < p.B && look(tid);
      if (__syncthreads_or(wrong)) b = -2;
      else b += __syncthreads_count(below);
    } else {
      int below = 0;
      for (int i = tid; i < p.B; i += kSelThreads) below += look(i) ? 1 : 0;
      below = __reduce_add_sync(0xffffffffu, below);
      if (lane == 0) red[0][warp][0] = below;
      if (__syncthreads_or(wrong)) b = -2;
      else {
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w) b += red[0][w][0];
      }
      __syncthreads();
    }
    if (b == -2) {
      if (tid == 0) atomicExch(p.status, DEV_BAD_OFFSETS);
      return;
    }
  }
  const Seq t(p, b);
  const int seen = t.seen(p, q - t.q0);
  int* out = p.out + unit * p.count;
  if (seen <= p.count) {
    for (int e = tid; e < p.count; e += kSelThreads) out[e] = e < seen ? e : -1;
    return;
  }
  for (int e = tid; e < p.first; e += kSelThreads) out[e] = e;
  for (int e = tid; e < p.last; e += kSelThreads) out[p.count - p.last + e] = seen - p.last + e;
  const int n = seen - p.first - p.last, k = p.count - p.first - p.last;   // k of n candidates
  if (k == 0) return;
  scores += p.first;
  float* v = in_smem ? local : scores;
  // ---- candidates and their range; NaN ranks above all
  int low_bits = 0x7fffffff, high_bits = -0x7fffffff - 1;
  float eps = 0.f;
  bool strange = false;
  for (int i = p.first / kStep + tid; i <= (seen - p.last - 1) / kStep; i += kSelThreads) eps = fmaxf(eps, p.errors[unit * p.groups + i]);
  for (int i = tid, a = 0; i < n; i += kSelThreads, ++a) {
    float x = a == 0 ? ahead[0] : a == 1 ? ahead[1] : a == 2 ? ahead[2] : a == 3 ? ahead[3] : scores[i];
    if (x != x) x = INFINITY;
    else {
      strange |= !(fabsf(x) <= kBig);
      low_bits = min(low_bits, ordered32(x));
      high_bits = max(high_bits, ordered32(x));
    }
    v[i] = x;
  }
  low_bits = __reduce_min_sync(0xffffffffu, low_bits);
  high_bits = __reduce_max_sync(0xffffffffu, high_bits);
  eps = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(eps)));
  if (lane == 0) redf[warp] = make_int4(low_bits, high_bits, __float_as_int(eps), 0);
  strange = __syncthreads_or(strange) != 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) {
    const int4 r = redf[w];
    low_bits = min(low_bits, r.x);
    high_bits = max(high_bits, r.y);
    eps = fmaxf(eps, __int_as_float(r.z));
  }
  float low = unordered32(low_bits), high = unordered32(high_bits);
  // Sums over all threads of two counts, and what the threads before this one have; every second call has its
  // own slots.
  int turn = 0;
  auto scan2 = [&](int a, int b2, int2& before) -> int2 {
    int ia = a, ib = b2;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int xa = __shfl_up_sync(0xffffffffu, ia, o), xb = __shfl_up_sync(0xffffffffu, ib, o);
      if (lane >= o) {
        ia += xa;
        ib += xb;
      }
    }
    if (lane == 31) {
      red[turn][warp][0] = ia;
      red[turn][warp][1] = ib;
    }
    __syncthreads();
    before = make_int2(ia - a, ib - b2);
    int2 sum = make_int2(0, 0);
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
      const int xa = red[turn][w][0], xb = red[turn][w][1];
      if (w < warp) {
        before.x += xa;
        before.y += xb;
      }
      sum.x += xa;
      sum.y += xb;
    }
    turn ^= 1;
    return sum;
  };
  // ---- the border: pages above `top` are among the k best for sure, those below `bottom` are not.  Of [low, high]
  // the k-th largest score is known to lie there: at least k are >= low, fewer than k above high.
  float top = INFINITY, bottom = -INFINITY;
  // None is sure where scores may have overflowed, or differ by less than the bins' arithmetic holds.
  const bool all = strange || !(eps <= kBig / 1048576.f) || (high - low > eps && high - low < 1e-30f);
  if (!all && low_bits > high_bits) {        // NaN pages only
    bottom = kBig;
  } else if (!all) {
    // Histograms of the range, which becomes the bin that holds the k-th largest until it is narrower than the error.
    bool found = false;
    for (int it = 0; it < 8 && !found; ++it) {
      int* hist = bins[it & 1];
      const float width = high - low, to_bin = width > 0.f ? kBins / width : 0.f;
      for (int i = tid; i < n; i += kSelThreads) {
        const float x = v[i];
        if (x > high) atomicAdd(hist + kBins, 1);
        else if (x >= low) atomicAdd(hist + min((int)((x - low) * to_bin), kBins - 1), 1);
      }
      __syncthreads();
      // Every warp looks: lane l has bins 8 l .. 8 l + 7.
      const int4 y = reinterpret_cast<const int4*>(hist)[2 * lane], z = reinterpret_cast<const int4*>(hist)[2 * lane + 1];
      const int c8[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w}, sum = ((y.x + y.y) + (y.z + y.w)) + ((z.x + z.y) + (z.z + z.w));
      int above = sum;                       // in this lane's bins and all higher ones
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_down_sync(0xffffffffu, above, o);
        if (lane + o < 32) above += x;
      }
      const int over = hist[kBins];
      above += over;
      if (over >= k) {                       // enough NaN pages to fill the list
        bottom = kBig;
        found = true;
        break;
      }
      const uint32_t votes = __ballot_sync(0xffffffffu, above >= k);
      const int owner = 31 - __clz(votes);   // (at least k are >= low)
      int bin = 0, run = above - sum;
#pragma unroll
      for (int i = 7; i >= 0; --i) {
        if (run < k && run + c8[i] >= k) bin = lane * 8 + i;
        run += c8[i];
      }
      bin = __shfl_sync(0xffffffffu, bin, owner);
      const float slack = width * 9.5367431640625e-7f;             // 2^-20: bins are found by rounded arithmetic
      const float lo2 = low + bin * (width / kBins) - slack, hi2 = low + (bin + 1) * (width / kBins) + slack;
      low = fmaxf(low, lo2);
      high = fminf(high, hi2);
      found = high - low <= eps || high - low >= width;
      if (!found) {                          // the other histogram is the next one; this one's turn comes after it
        __syncthreads();
        hist[tid] = 0;
        if (tid == 0) hist[kBins] = 0;
      }
    }
    if (bottom != kBig) {
      // Twice the error, and a few roundings of the bins' borders, which are far below it.
      top = high + 2.1f * eps;
      bottom = low - 2.1f * eps;
    }
  }
  // ---- thread t has candidates [t per, ...): sure ones and those near the border
  const int per = (n + kSelThreads - 1) / kSelThreads, mine_lo = min(tid * per, n), mine_hi = min(mine_lo + per, n);
  int in = 0, near = 0;
  for (int i = mine_lo; i < mine_hi; ++i) {
    const float x = v[i];
    if (x > top) ++in;
    else if (x >= bottom) ++near;
  }
  int2 before;
  const int2 both = scan2(in, near, before);
  const int need = k - both.x, m = both.y;   // of the m pages near the border
  int place = before.x + before.y;
  float emit = bottom;                       // listed: v >= emit
  if (m != need) {
    // ---- these exactly, in the order of their numbers
    unsigned long long* keys = m <= kFew ? few_keys : p.exact + unit * p.max_pages;
    int* at = m <= kFew ? few_at : p.near + unit * p.max_pages;
    for (int i = mine_lo, x = before.y; i < mine_hi; ++i)
      if (!(v[i] > top) && v[i] >= bottom) {
        keys[x] = 0;                         // below every number
        at[x++] = i;
      }
    __syncthreads();
    const int* table = p.table + (long long)b * p.max_pages + p.first;
    // A warp takes a few heads of a page; the largest of them all counts.
    const long long shares = (p.g + kExactHeads - 1) / kExactHeads;
    for (long long a = warp; a < m * shares; a += kSelWarps) {
      const int near_at = (int)(a / shares), r0 = (int)(a - near_at * shares) * kExactHeads, pg = __ldg(table + at[near_at]);
      unsigned long long key = 1ull << 63;   // 0
      if (eps != 0.f && pg >= 0 && pg < p.num_pages) key = exact_score<D>(p, q, h, r0, pg);   // (eps = 0: q is, or the scales)
      if (lane == 0) atomicMax(keys + near_at, key);
    }
    __syncthreads();
    if (m <= kFew) {
      if (tid < m) {                         // rank: better ones, and equal ones before it
        const unsigned long long mine = keys[tid];
        int better = 0;
        for (int a = 0; a < m; ++a) better += keys[a] > mine || (keys[a] == mine && a < tid) ? 1 : 0;
        v[at[tid]] = better < need ? INFINITY : -INFINITY;
      }
    } else {
      // The need-th largest key, bit by bit; then of the keys equal to it the first ones.
      int2 unused;
      unsigned long long key = 0;
      for (int bit = 63; bit >= 0; --bit) {
        const unsigned long long trial = key | (1ull << bit);
        int enough = 0;
        for (int a = tid; a < m; a += kSelThreads) enough += keys[a] >= trial ? 1 : 0;
        if (scan2(enough, 0, unused).x >= need) key = trial;
      }
      const int per_key = (m + kSelThreads - 1) / kSelThreads, a_lo = min(tid * per_key, m), a_hi = min(a_lo + per_key, m);
      int better = 0, equal = 0;
      for (int a = a_lo; a < a_hi; ++a) {
        better += keys[a] > key ? 1 : 0;
        equal += keys[a] == key ? 1 : 0;
      }
      int2 ahead_of;
      const int equal_need = need - scan2(better, equal, ahead_of).x;
      for (int a = a_lo, x = ahead_of.y; a < a_hi; ++a) {
        const bool take = keys[a] > key || (keys[a] == key && x++ < equal_need);
        v[at[a]] = take ? INFINITY : -INFINITY;
      }
    }
    __syncthreads();
    emit = fminf(top, kBig);                 // the chosen ones are infinite now, the others -inf
    if (top < kBig) emit = nextafterf(top, INFINITY);
    in = 0;
    for (int i = mine_lo; i < mine_hi; ++i) in += v[i] >= emit ? 1 : 0;
    scan2(in, 0, before);
    place = before.x;
  }
  // ---- out, ascending
  for (int i = mine_lo; i < mine_hi; ++i)
    if (v[i] >= emit && place < k) out[p.first + place++] = p.first + i;
}

}  // namespace

// [Hkv][total_q] rows: scores, the exact keys and numbers of pages near the border, the steps' errors.
SelectWs select_ws(int Hkv, int total_q, int max_pages) {
  const auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  const size_t rows = (size_t)Hkv * total_q, groups = ((size_t)max_pages + kStep - 1) / kStep;
  SelectWs w;
  w.exact = up(rows * max_pages * 4);
  w.near = w.exact + up(rows * max_pages * 8);
  w.errors = w.near + up(rows * max_pages * 4);
  w.total = w.errors + up(rows * groups * 4);
  return w;
}

cudaError_t launch_select_pages(SelectParams p, int d, int sms, cudaStream_t s) {
  p.page_shift = p.page == 16 ? 4 : p.page == 32 ? 5 : p.page == 64 ? 6 : 7;
  // Queries of a tile: as many as fill 16 rows (8 rows, when all of a sequence's fit), but no more than it has.
  const bool small = (long long)p.max_q * p.g <= 8;
  p.qn = p.g >= 16 ? 1 : (p.max_q < 16 / p.g ? p.max_q : 16 / p.g);
  p.groups = (p.max_pages + kStep - 1) / kStep;
  const long long lists = (long long)p.total_q * p.Hkv;            // below 2^31
  cudaError_t e = cudaSuccess;
  const dim3 grid((unsigned)(kScoreCtas * sms));
  auto score = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(kScoreThreads), 0, s, p); };
  if (p.max_pages > p.count) {               // (else every list holds all pages)
    if (d == 64) e = small ? score(select_score_kernel<64, 1>) : score(select_score_kernel<64, 2>);
    else e = small ? score(select_score_kernel<128, 1>) : score(select_score_kernel<128, 2>);
  }
  if (e != cudaSuccess) return e;
  const size_t bytes = (size_t)p.max_pages * 4;
  const int in_smem = bytes <= 40 * 1024 ? 1 : 0;      // (longer tables: in the workspace)
  return d == 64 ? launch_pdl(select_choose_kernel<64>, dim3((unsigned)lists), dim3(kSelThreads), in_smem ? bytes : 0, s, p, in_smem)
                 : launch_pdl(select_choose_kernel<128>, dim3((unsigned)lists), dim3(kSelThreads), in_smem ? bytes : 0, s, p, in_smem);
}

}  // namespace attn
