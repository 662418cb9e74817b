// New K and V rows into a paged e4m3 cache, K rotated on the way, and bounds of each page's keys.
//
// Page scales, codes and slots are kv_append.cu's.  K differs in what is coded: with the rotation
// of rope.cu in fp32, y = R(pos) x, the page's largest finite |y| sets the scale and code =
// e4m3(y / s).  Rotated rows are never rounded to bf16 in between, nor do they cross memory.
// Bounds: per page, K/V head and column the smallest and the largest code of the page's rows (a
// NaN code where a column holds one), which a choice of pages to read goes by.  Codes of earlier
// rows that are rounded again at a grown scale keep their order, so the bounds kept with them are
// rounded the same way and stay exact, without a look at the rows.
//
// Bound by bytes (2 read, 1 written per element); what must not show is the sines and cosines, one
// pair per token and two columns, the same for all heads (with a CTA per head, each making its own, K and V of the prompts below took 58 us, 36 now).
// Two kernels:
//   * few rows per sequence or page: a CTA per slot, 8 heads and K or V, a warp per head.  The CTA
//     fills a table of 16 rows' sines and cosines, so each is made once for 8 heads.  One row of 64
//     sequences, 32 + 8 heads: 5.7 us in a graph, queries included;
//   * prompts: a CTA per slot, up to 8 heads and K or V.  The page's table is made while the first
//     head's rows are on their way from memory; a head's rotated rows are kept in fp32 between the
//     maximum and the rounding, and the next head's are under way meanwhile.  That is more than the registers
//     hold: of a thread's 364 bytes are stored and 420 loaded in local memory with pages of 128 and d = 128 (128
//     registers), about 230 and 310 with 16 elements a thread at 64 registers, 36 to 96 elsewhere.  V goes through the
//     same kernel, whose registers and table it does not need.  Two prompts of 8192, 32 + 8 heads, d = 128: 74 us with
//     the queries' 42 (5.0 TB/s), K and V alone 36; attn_rope and attn_kv_append_fp8 one after the other take
//     72, so with prompts the call saves a rounding of K and keeps bounds, but no time.
// The queries rotate in the same launch where there are few of them, else in rope.cu's kernel, beside this one where
// it leaves room.
#include <cstdint>
#include <mutex>

#include "append.cuh"
#include "rope.cuh"

namespace attn {
namespace {

// How K's columns turn: not at all; halves, neighbours (rot a multiple of 8); any even rot.
enum : int { TURN_NONE = 0, TURN_SPLIT = 1, TURN_INTER = 2, TURN_ANY = 3 };
__device__ __forceinline__ int turn_mode(const RopeAppendParams& p, bool is_v) {
  if (is_v || p.rot == 0) return TURN_NONE;
  return p.rot % 8 != 0 ? TURN_ANY : p.interleaved ? TURN_INTER : TURN_SPLIT;
}
// Where pair j's (cos, sin) lies in a row of the table: 16-byte pieces (two pairs) that the threads of a
// row read at the same time lie side by side.
template <int mode>
__device__ __forceinline__ int turn_slot(int rot, int j) {
  const int f = j >> 1;
  if (mode == TURN_SPLIT) {                  // groups of 4 columns: pairs 4 g .. 4 g + 3, two pieces
    const int g = f >> 1;
    return (((f & 1) * 2 + (g & 1)) * ((rot / 8 + 1) / 2) + (g >> 1)) * 2 + (j & 1);
  }
  if (mode == TURN_INTER) return ((f & 1) * (rot / 8) + (f >> 1)) * 2 + (j & 1);
  return j;
}
// Pairs that a row of the table has room for.
__host__ __device__ inline int turn_row(int rot) { return rot % 8 == 0 ? (rot / 8 + 1) / 2 * 8 : rot / 2; }
// Rows r .. r + n - 1 of the slot's page into the table, by all threads: a thread has one pair of every few rows.
template <int mode, int THREADS>
__device__ __forceinline__ void fill_turns(const RopeAppendParams& p, const Slot& s, int r, int n,
                                           const unsigned long long* turn, float2* cs) {
  const int half = p.rot / 2, stride = turn_row(p.rot), step = THREADS / half;     // (half <= 64)
  const int row0 = threadIdx.x / half, j = threadIdx.x - row0 * half;
  if (row0 >= step) return;
  const unsigned long long t = turn[j];
  float2* out = cs + turn_slot<mode>(p.rot, j);
#pragma unroll 2
  for (int row = row0; row < n; row += step) {
    const long long pos = p.positions ? __ldg(p.positions + s.src0 + r + row) : s.first + r + row;
    float sn, c;
    turn_sincos_near(t, pos, sn, c);
    out[row * stride] = make_float2(c * p.mscale, sn * p.mscale);
  }
}

// Columns 8 c .. 8 c + 7 of a row, rotated: own are they, row the whole row in memory (TURN_ANY), cs the
// row's sines and cosines.  All lanes of a warp call it together; lane holds column group c of its row.
template <int mode>
__device__ __forceinline__ void turned(const RopeAppendParams& p, const uint4& own, const uint16_t* row, int c,
                                       const float2* cs, float (&y)[8]) {
  bf16x8(own, y);
  const int rot = p.rot;
  if constexpr (mode == TURN_NONE) {
  } else if constexpr (mode == TURN_SPLIT) {
    // Four columns at a time: group g of the first half turns with g + q, whose lane and whose place there (one
    // for all lanes) follow.
    const int q = rot / 8, lane = threadIdx.x & 31, width = (q + 1) / 2;
    const float4* table = reinterpret_cast<const float4*>(cs);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int g = 2 * c + k;
      const bool upper = g >= q, turns = g < 2 * q;
      const int other = turns ? (upper ? g - q : g + q) : g, from = lane - c + (other >> 1);
      const bool odd = ((k + q) & 1) != 0;
      const uint32_t a = __shfl_sync(0xffffffffu, odd ? own.z : own.x, from), b = __shfl_sync(0xffffffffu, odd ? own.w : own.y, from);
      if (!turns) continue;
      const int pair = upper ? other : g;    // group of pairs
      const float z[4] = {__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u), __uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u)};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 e = table[(i * 2 + (pair & 1)) * width + (pair >> 1)];
        const int x = 4 * k + 2 * i;
        y[x] = turn_one(y[x], z[2 * i], e.x, e.y, upper);
        y[x + 1] = turn_one(y[x + 1], z[2 * i + 1], e.z, e.w, upper);
      }
    }
  } else if constexpr (mode == TURN_INTER) {
    if (8 * c >= rot) return;
    const float4* at = reinterpret_cast<const float4*>(cs) + c;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float4 e = at[q * (rot / 8)];
      const float a = y[4 * q], b = y[4 * q + 1], d = y[4 * q + 2], f = y[4 * q + 3];
      turn_pair(a, b, e.x, e.y, y[4 * q], y[4 * q + 1]);
      turn_pair(d, f, e.z, e.w, y[4 * q + 2], y[4 * q + 3]);
    }
  } else {
    const int half = rot / 2;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int col = 8 * c + k;
      if (col >= rot) continue;
      const bool second = p.interleaved ? (col & 1) != 0 : col >= half;
      const int j = p.interleaved ? col >> 1 : (second ? col - half : col);
      const int other = p.interleaved ? col ^ 1 : (second ? col - half : col + half);
      const float z = __uint_as_float((uint32_t)__ldg(row + other) << 16);
      const float2 e = cs[j];
      y[k] = turn_one(y[k], z, e.x, e.y, second);
    }
  }
}

// Rows are rotated once for their maximum and once more for their codes; left to itself the compiler keeps the
// first results in local memory instead.
template <int N>
__device__ __forceinline__ void forget(uint4 (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(x[i].x), "+r"(x[i].y), "+r"(x[i].z), "+r"(x[i].w));
}

// Largest finite |y|; where an infinity hides it (a maximum passes NaN by), they are looked at one by one.
__device__ __forceinline__ float largest8(const float (&y)[8], float m) {
#pragma unroll
  for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(y[k]));
  return m;
}
__device__ __noinline__ float largest_finite8(float4 a, float4 b) {
  const float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = fabsf(y[k]) < INFINITY ? fmaxf(m, fabsf(y[k])) : m;
  return m;
}
__device__ __forceinline__ float finite8(const float (&y)[8], float m) {
  return fmaxf(m, largest_finite8(make_float4(y[0], y[1], y[2], y[3]), make_float4(y[4], y[5], y[6], y[7])));
}
// (inv = 0: a scale that is no power of two, by division.)
__device__ __noinline__ uint2 divided8(float4 a, float4 b, float scale) {
  const float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float f[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = __fdiv_rn(y[k], scale);
  return e4m3x8(f);
}
__device__ __forceinline__ uint2 coded8(const float (&y)[8], float inv, float scale) {
  if (inv == 0.f) return divided8(make_float4(y[0], y[1], y[2], y[3]), make_float4(y[4], y[5], y[6], y[7]), scale);
  float f[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = y[k] * inv;
  return e4m3x8(f);
}

// Smallest and largest of codes, column by column, in f16 (which holds every e4m3 value); NaN wins.
struct Bounds {
  __half2 lo[4], hi[4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = __float2half2_rn(INFINITY);
      hi[i] = __float2half2_rn(-INFINITY);
    }
  }
  static __device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
  __device__ __forceinline__ void add(const uint2& low, const uint2& high) {
    const uint32_t l[4] = {e4m3x2_f16x2(low.x), e4m3x2_f16x2_hi(low.x), e4m3x2_f16x2(low.y), e4m3x2_f16x2_hi(low.y)};
    const uint32_t h[4] = {e4m3x2_f16x2(high.x), e4m3x2_f16x2_hi(high.x), e4m3x2_f16x2(high.y), e4m3x2_f16x2_hi(high.y)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = __hmin2_nan(lo[i], as_half2(l[i]));
      hi[i] = __hmax2_nan(hi[i], as_half2(h[i]));
    }
  }
  __device__ __forceinline__ void add(const Bounds& b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = __hmin2_nan(lo[i], b.lo[i]);
      hi[i] = __hmax2_nan(hi[i], b.hi[i]);
    }
  }
  // Over the lanes that hold the same columns of other rows (D / 8 lanes per row).
  __device__ __forceinline__ void over_rows(int lanes_per_row) {
    for (int o = lanes_per_row; o < 32; o <<= 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] = __hmin2_nan(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
        hi[i] = __hmax2_nan(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
      }
    }
  }
  static __device__ __forceinline__ uint2 codes(const __half2 (&x)[4]) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint16_t c;
      asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(*reinterpret_cast<const uint32_t*>(&x[i])));
      r[i] = c;
    }
    return make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
  }
  // With the bounds of the earlier rows, whose codes became recode8(code, s_old, inv) if the scale grew.
  __device__ __forceinline__ void store(uint8_t* page, int d, int c, bool earlier, bool grown, float s_old, float inv) {
    uint2* low = reinterpret_cast<uint2*>(page + c * 8);
    uint2* high = reinterpret_cast<uint2*>(page + d + c * 8);
    if (earlier) {
      const uint2 l = *low, h = *high;
      add(grown ? recode8(l, s_old, inv) : l, grown ? recode8(h, s_old, inv) : h);
    }
    *low = codes(lo);
    *high = codes(hi);
  }
};

constexpr int kStepWarps = 8, kStepRows = 16;          // rows of the table

// A slot's page of 8 heads of K or V, a warp per head.
template <int D, int mode>
__device__ __forceinline__ void append_step(const RopeAppendParams& p, const Slot& s, bool is_v, const unsigned long long* turn,
                                            float2* cs) {
  constexpr int THREADS = kStepWarps * 32, LPR = D / 8, RPW = 32 / LPR, STEPS = kStepRows / RPW;   // lanes per row, rows at once
  const int lane = threadIdx.x & 31, head = blockIdx.x / (2 * p.slots) * kStepWarps + (threadIdx.x >> 5);
  const int stride = turn_row(p.rot);
  const bool live = head < p.a.Hkv;
  const Target t(p.a, s, live ? head : 0, is_v, D);
  const int r0 = lane / LPR, c = lane % LPR;
  const float s_old = s.kept > 0 && live ? *t.scale : 0.f;
  uint4 x[STEPS];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int r = base + i * RPW + r0;
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (live && r < s.rows) x[i] = *reinterpret_cast<const uint4*>(t.src + (s.src0 + r) * t.st + c * 8);
    }
  };
  auto table = [&](int base) {                         // after the loads: they are under way meanwhile
    if (mode == TURN_NONE) return;
    __syncthreads();                                   // the rows before have been used
    fill_turns<mode, THREADS>(p, s, base, min(kStepRows, s.rows - base), turn, cs);
    __syncthreads();
  };
  auto row = [&](int base, int i, float (&y)[8]) {
    const int r = min(i * RPW + r0, s.rows - base - 1);          // (lanes without a row: any one, as 0)
    turned<mode>(p, x[i], t.src + (s.src0 + base + r) * t.st, c, cs + r * stride, y);
  };
  const bool one = s.rows - s.kept <= kStepRows;       // the rows and the table are kept for the second pass
  float amax = 0.f;
  for (int base = s.kept; base < s.rows; base += kStepRows) {
    load(base);
    table(base);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      if (base + i * RPW >= s.rows) break;
      float y[8];
      row(base, i, y);
      if (base + i * RPW + r0 < s.rows) m = largest8(y, m);
    }
    if (__any_sync(0xffffffffu, m == INFINITY)) {
      m = 0.f;
#pragma unroll 1
      for (int r = 0; r < kStepRows; r += RPW) {
        uint4 w = x[0];
#pragma unroll
        for (int i = 1; i < STEPS; ++i)
          if (r == i * RPW) w = x[i];
        float y[8];
        turned<mode>(p, w, t.src + (s.src0 + min(base + r + r0, s.rows - 1)) * t.st, c, cs + min(r + r0, s.rows - base - 1) * stride, y);
        if (base + r + r0 < s.rows) m = finite8(y, m);
      }
    }
    amax = fmaxf(amax, m);
  }
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  const float sc = fmaxf(s_old, pow2_scale(amax));
  const float inv = exact_inverse(sc);
  const bool keep_bounds = p.bounds != nullptr && !is_v;
  Bounds b;
  b.clear();
  forget(x);
  for (int base = s.kept; base < s.rows; base += kStepRows) {
    if (!one) {
      load(base);
      table(base);
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      if (base + i * RPW >= s.rows) break;
      float y[8];
      row(base, i, y);
      const int r = base + i * RPW + r0;
      if (!live || r >= s.rows) continue;
      const uint2 code = coded8(y, inv, sc);
      *reinterpret_cast<uint2*>(t.dst + r * D + c * 8) = code;
      if (keep_bounds) b.add(code, code);
    }
  }
  if (!live) return;                                   // (whole warps; no barrier follows)
  if (sc > s_old) {
    for (int r = r0; r < s.kept; r += RPW) {
      uint2* out = reinterpret_cast<uint2*>(t.dst + r * D + c * 8);
      *out = recode8(*out, s_old, inv);
    }
  }
  if (keep_bounds) {
    b.over_rows(LPR);
    if (r0 == 0) b.store(p.bounds + ((long long)s.page * p.a.Hkv + head) * 2 * D, D, c, s.kept > 0, sc > s_old, s_old, inv);
  }
  __syncwarp();                                        // every lane has read the old scale
  if (lane == 0) *t.scale = sc;
}

// The queries of packed row t, rotated as rope.cu's kernel does (the same bits); few rows only.
template <int D, int mode>
__device__ __forceinline__ void turn_queries(const RopeAppendParams& p, int t, const unsigned long long* turn, float2* cs) {
  constexpr int THREADS = kStepWarps * 32, LPR = D / 8, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, r0 = lane / LPR, c = lane % LPR;
  const int h0 = (threadIdx.x >> 5) * RPW;             // this warp's first heads
  const uint16_t* src = static_cast<const uint16_t*>(p.q) + t * p.q_t + c * 8;
  uint16_t* dst = static_cast<uint16_t*>(p.q_out) + t * p.o_t + c * 8;
  auto load = [&](int h) -> uint4 {
    return h + r0 < p.Hq ? *reinterpret_cast<const uint4*>(src + (h + r0) * p.q_h) : make_uint4(0u, 0u, 0u, 0u);
  };
  uint4 x = load(h0);
  long long pos;
  if (p.positions) {
    pos = __ldg(p.positions + t);
  } else {                                             // the last sequence that starts at or before it
    int b = -1;
    for (int i = 0; i < p.a.B; i += THREADS) b += __syncthreads_count(i + threadIdx.x < p.a.B && __ldg(p.a.cu + min(i + (int)threadIdx.x, p.a.B - 1)) <= t);
    b = max(b, 0);                                     // (invalid offsets only make it wrong)
    pos = (long long)__ldg(p.a.kv_lens + b) - __ldg(p.a.cu + b + 1) + t;
  }
  __syncthreads();                                     // turn
  for (int j = threadIdx.x; j < p.rot / 2; j += THREADS) {
    float sn, co;
    turn_sincos(turn[j], pos, sn, co);
    cs[turn_slot<mode>(p.rot, j)] = make_float2(co * p.mscale, sn * p.mscale);
  }
  __syncthreads();
  for (int h = h0; h < p.Hq; h += kStepWarps * RPW) {
    const uint4 now = x;
    x = load(h + kStepWarps * RPW);
    float y[8];
    turned<mode>(p, now, nullptr, c, cs, y);
    if (h + r0 < p.Hq)
      *reinterpret_cast<uint4*>(dst + (h + r0) * p.o_h) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
  }
}

// Block x: of the first 2 slots x head groups, slot x / 2 mod slots, K or V by x & 1, 8 heads a group; behind
// them the queries of a row each.
template <int D>
__global__ void __launch_bounds__(kStepWarps * 32) rope_append_step_kernel(const RopeAppendParams p) {
  __shared__ unsigned long long turn[D / 2];
  __shared__ __align__(16) float2 cs[kStepRows * D / 2];         // (a row of the table: at most D / 2 pairs)
  constexpr int THREADS = kStepWarps * 32;
  pdl_trigger();                                       // the queries' rotation may start
  const int kv_blocks = 2 * p.slots * ((p.a.Hkv + kStepWarps - 1) / kStepWarps), x = blockIdx.x % (2 * p.slots);
  const bool queries = (int)blockIdx.x >= kv_blocks, is_v = !queries && (x & 1);
  const int mode = turn_mode(p, is_v);
  if (mode != TURN_NONE)
    for (int j = threadIdx.x; j < p.rot / 2; j += THREADS) turn[j] = turns_per_position(p.inv_freq[j]);
  if (queries) {
    if (mode == TURN_SPLIT) turn_queries<D, TURN_SPLIT>(p, (int)blockIdx.x - kv_blocks, turn, cs);
    else turn_queries<D, TURN_INTER>(p, (int)blockIdx.x - kv_blocks, turn, cs);
    return;
  }
  Slot s;
  if (!find_slot<THREADS>(p.a, x >> 1, s)) return;     // (its barrier stands behind the writes of turn)
  if (mode == TURN_NONE) append_step<D, TURN_NONE>(p, s, is_v, turn, cs);
  else if (mode == TURN_SPLIT) append_step<D, TURN_SPLIT>(p, s, is_v, turn, cs);
  else if (mode == TURN_INTER) append_step<D, TURN_INTER>(p, s, is_v, turn, cs);
  else append_step<D, TURN_ANY>(p, s, is_v, turn, cs);
}

// A slot's page of p.heads_per_cta heads of K or V by a CTA: 8 elements per thread and step, NV steps cover a
// head's.  The next head's rows are under way while one is worked on.
template <int D, int NV, int THREADS, int mode>
__device__ __forceinline__ void append_page(const RopeAppendParams& p, const Slot& s, bool is_v, const unsigned long long* turn,
                                            float2* cs, uint32_t* red, Bounds (*parts)[D / 8]) {
  constexpr int LPR = D / 8, RPS = THREADS / LPR;      // lanes per row, rows per step
  const int tid = threadIdx.x, stride = turn_row(p.rot), r0 = tid / LPR, c = tid % LPR;
  const int h_begin = blockIdx.y * p.heads_per_cta, h_end = min(h_begin + p.heads_per_cta, p.a.Hkv);
  uint4 ahead[NV];
  auto load = [&](const Target& t) {
    const uint16_t* src = t.src + (s.src0 + r0) * t.st + c * 8;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int r = r0 + i * RPS;
      ahead[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r >= s.kept && r < s.rows) ahead[i] = *reinterpret_cast<const uint4*>(src + i * RPS * t.st);
    }
  };
  load(Target(p.a, s, h_begin, is_v, D));
  if (mode != TURN_NONE) {
    fill_turns<mode, THREADS>(p, s, s.kept, s.rows - s.kept, turn, cs);
    __syncthreads();
  }
  const bool keep_bounds = p.bounds != nullptr && !is_v;
#pragma unroll 1
  for (int head = h_begin; head < h_end; ++head) {
    const Target t(p.a, s, head, is_v, D);
    const float s_old = s.kept > 0 ? *t.scale : 0.f;
    // The rotated rows are kept until the page's scale is known.
    float y[NV][8], amax = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {                     // (threads without a row: any one, as 0)
      const int r = max(min(r0 + i * RPS, s.rows - 1), s.kept);
      turned<mode>(p, ahead[i], t.src + (s.src0 + r) * t.st, c, cs + (r - s.kept) * stride, y[i]);
      amax = largest8(y[i], amax);                     // (a row read as 0 stays 0, but for TURN_ANY: below)
    }
    if (head + 1 < h_end) load(Target(p.a, s, head + 1, is_v, D));
    if (amax == INFINITY || mode == TURN_ANY) {
      amax = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int r = r0 + i * RPS;
        if (r >= s.kept && r < s.rows) amax = finite8(y[i], amax);
      }
    }
    uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
    if ((tid & 31) == 0) red[(head & 1) * (THREADS / 32) + (tid >> 5)] = bits;     // (every second head its own: one barrier)
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) bits = max(bits, red[(head & 1) * (THREADS / 32) + i]);
    const float sc = fmaxf(s_old, pow2_scale(__uint_as_float(bits)));
    if (tid == 0) *t.scale = sc;                       // (all have read the old one before the barrier)
    const float inv = exact_inverse(sc);
    Bounds b;
    b.clear();
    uint2* out = reinterpret_cast<uint2*>(t.dst + tid * 8);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int r = r0 + i * RPS;                      // rows behind the last one stay as they are
      if (r < s.kept || r >= s.rows) continue;
      const uint2 code = coded8(y[i], inv, sc);
      out[i * THREADS] = code;
      if (keep_bounds) b.add(code, code);
    }
    if (sc > s_old) {                                  // the kept rows' codes change (under a scale of 0: to 0)
#pragma unroll 1
      for (int i = 0; i < NV && r0 + i * RPS < s.kept; ++i) out[i * THREADS] = recode8(out[i * THREADS], s_old, inv);
    }
    if (keep_bounds) {
      b.over_rows(LPR);
      if (head > h_begin) __syncthreads();             // the parts before have been read
      if ((tid & 31) < LPR) parts[tid >> 5][c] = b;
      __syncthreads();
      if (tid < LPR) {
        for (int w = 1; w < THREADS / 32; ++w) b.add(parts[w][tid]);
        b.store(p.bounds + ((long long)s.page * p.a.Hkv + head) * 2 * D, D, tid, s.kept > 0, sc > s_old, s_old, inv);
      }
    }
  }
}

// Block: slot x, heads y, K or V z.
template <int D, int NV, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) rope_append_kernel(const RopeAppendParams p) {
  extern __shared__ __align__(16) float2 cs[];         // [new rows][turn_row]
  __shared__ unsigned long long turn[D / 2];
  __shared__ uint32_t red[2 * (THREADS / 32)];
  __shared__ Bounds parts[THREADS / 32][D / 8];
  pdl_trigger();                                       // the queries' rotation may start
  const bool is_v = blockIdx.z != 0;
  const int mode = turn_mode(p, is_v);
  if (mode != TURN_NONE)
    for (int j = threadIdx.x; j < p.rot / 2; j += THREADS) turn[j] = turns_per_position(p.inv_freq[j]);
  Slot s;
  if (!find_slot<THREADS>(p.a, blockIdx.x, s)) return; // (its barrier stands behind the writes of turn)
  if (mode == TURN_NONE) append_page<D, NV, THREADS, TURN_NONE>(p, s, is_v, turn, cs, red, parts);
  else if (mode == TURN_SPLIT) append_page<D, NV, THREADS, TURN_SPLIT>(p, s, is_v, turn, cs, red, parts);
  else if (mode == TURN_INTER) append_page<D, NV, THREADS, TURN_INTER>(p, s, is_v, turn, cs, red, parts);
  else append_page<D, NV, THREADS, TURN_ANY>(p, s, is_v, turn, cs, red, parts);
}

template <int D>
cudaError_t launch_d(const RopeAppendParams& p, dim3 grid, cudaStream_t s) {
  const int vecs = p.a.page * D / 8;                   // 16-byte pieces of a page
  const size_t smem = (size_t)p.a.page * turn_row(p.rot) * sizeof(float2);
  if constexpr (D == 64) {
    if (vecs == 128) rope_append_kernel<D, 1, 128, 8><<<grid, 128, smem, s>>>(p);
  } else if (vecs == 2048) {
    // The only table of more than 40 KB (a page of 128: 64 KB).
    static std::once_flag flags[64];
    static cudaError_t attr_err[64];
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::call_once(flags[dev & 63], [&] {
      attr_err[dev & 63] = cudaFuncSetAttribute(rope_append_kernel<D, 8, 256, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * D / 2 * 8);
    });
    if (attr_err[dev & 63] != cudaSuccess) return attr_err[dev & 63];
    rope_append_kernel<D, 8, 256, 2><<<grid, 256, smem, s>>>(p);
  }
  if (vecs == 256) rope_append_kernel<D, 1, 256, 4><<<grid, 256, smem, s>>>(p);
  else if (vecs == 512) rope_append_kernel<D, 2, 256, 4><<<grid, 256, smem, s>>>(p);
  else if (vecs == 1024) rope_append_kernel<D, 4, 256, 2><<<grid, 256, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_append(RopeAppendParams p, int d, int sms, bool* queries, cudaStream_t s) {
  const bool want = *queries;
  *queries = false;
  p.a.page_shift = p.a.page == 16 ? 4 : p.a.page == 32 ? 5 : p.a.page == 64 ? 6 : 7;
  const long long slots = (long long)p.a.total / p.a.page + 2LL * p.a.B;
  if (slots > 0x3fffffffLL || p.a.Hkv > 65535) return cudaErrorInvalidValue;
  // Up to 4 rows per sequence on average, and pages that get less than half their rows, a warp per page and head;
  // so that every SM has work (as in kv_append.cu): 256 pieces of 16 rows over pages of 64 / 128, 32 + 8 heads,
  // d = 128, 25 / 26 us against 37 / 54 with a CTA per page and heads.  Whole pages take CTAs, whatever their size (two
  // prompts of 8192: pages of 32 74 against 84; of 16 with d = 64 28 against 40, with d = 128 84 against 80).
  const bool small = 2LL * p.a.total <= slots * p.a.page && 2 * slots * p.a.Hkv >= 16LL * sms;
  if (p.a.total <= 4LL * p.a.B || small) {
    // A few rows' queries in the same launch (a token each of 64 sequences: 5.8 us in a graph either way, but 2.4 us
    // less of the host's time).
    *queries = want && p.a.total <= 4 * sms;
    p.slots = (int)slots;
    const long long grid = 2 * slots * ((p.a.Hkv + kStepWarps - 1) / kStepWarps) + (*queries ? p.a.total : 0);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (d == 64) rope_append_step_kernel<64><<<(unsigned)grid, kStepWarps * 32, 0, s>>>(p);
    else rope_append_step_kernel<128><<<(unsigned)grid, kStepWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
  }
  // Heads per CTA: as many as leave every SM work (the table is made once for them).
  p.heads_per_cta = 1;
  while (p.heads_per_cta < p.a.Hkv && p.heads_per_cta < 8 &&
         2 * slots * ((p.a.Hkv + 2 * p.heads_per_cta - 1) / (2 * p.heads_per_cta)) >= 3LL * sms)
    p.heads_per_cta *= 2;
  const dim3 grid((unsigned)slots, (unsigned)((p.a.Hkv + p.heads_per_cta - 1) / p.heads_per_cta), 2);
  return d == 64 ? launch_d<64>(p, grid, s) : launch_d<128>(p, grid, s);
}

}  // namespace attn
