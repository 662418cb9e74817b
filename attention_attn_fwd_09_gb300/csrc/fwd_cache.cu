// Attention of packed queries over a paged e4m3 cache: few query rows per K/V head (decoding,
// drafts of a few tokens).  Up to 16 rows, the n queries x g heads that share a K/V head, are
// one row tile (row r: query r / g, head r % g); the work is the cache, read once.
//
// What bounds it: the cache's bytes (2 d per key and K/V head).  So
//   * Work is cut by keys, not by sequences: all units (sequence, K/V head) laid end to end in
//     32-key pieces, every CTA takes the same number of consecutive pieces (lengths differ and
//     are known on the device only: each CTA adds them up itself).  A unit cut between CTAs
//     leaves partial results that fwd_cache_merge_kernel joins.
//   * A CTA has 4 warps and an SM two CTAs; each warp is on its own: it takes every fourth
//     piece, keeps a ring of pieces in flight with TMA (96 KB per CTA) and never waits for the
//     other warps until a unit ends.
//   * A piece goes from shared memory to registers in the layout the matrix instruction wants:
//     S = Q K^T and O += P V with mma.m16n8k16 in f16.  e4m3 widens to f16 exactly.  Both key
//     and column orders inside a piece are free (a sum does not mind, as long as P and V, or Q
//     and K, agree), which turns every fragment into whole 16-byte loads: a thread's share of a
//     K row is 16 neighbouring columns, its share of V 16 neighbouring columns of a key, and
//     pairs of keys are interleaved by byte permutes.  The key order within 8 (d = 128) or 16
//     (d = 64) rows is chosen so that under TMA's 128-byte swizzle both kinds of load touch
//     every bank once.
//
// Measured (d = 128, 32 heads on 8, one query): 64 sequences of up to 32768 keys 355 us, 6.2 TB/s of
// cache, 91 % of a copy's rate; 8 of 8192 keys 32.9 us in a graph, 4.1 TB/s (15 us of it are the
// start, the first pieces' way from memory and the merge); one of 1000 keys 8.6 us in a graph.
// With d = 64 (half the bytes, as many scores) the same take 0.78, 0.76 and 0.98 of these times.
//
// Numbers: q is scaled by a power of two per row (largest |q| in [2^14, 2^15)) and held in f16: exact
// down to 2^-31 of the row's largest component, off by at most 2^-39 of it below.  exp2(s - m + 14)
// <= 2^14 times the page's V scale over the largest V scale so far is rounded to f16 (11 bits, against
// 8 of a bf16 weight; the 2^14 keeps weights down to 2^-28 of the largest normal).  Scores, maxima,
// sums and O are fp32.
#include <cstdint>
#include <mutex>

#include "cache.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kPiece = 32;                   // keys per piece
constexpr int kSMs = 152;                  // blocks of the merge kernel are a multiple of these
constexpr float kShift = 14.f;               // weights are held times 2^14

template <int D>
struct DecCfg {
  static constexpr int KB = kPiece * D;            // bytes of a piece of K (and of V)
  static constexpr int STAGES = D == 128 ? 3 : 6;  // pieces per warp: 24 KB
  static constexpr int RING = kWarps * STAGES * 2 * KB;
  static constexpr int NACC = D / 8;               // O column blocks of 8
  static constexpr int SLOT = 32 * 4 * (NACC * 4); // one warp's O registers
  static constexpr int OFF_MERGE = RING;
  static constexpr int OFF_STAT = OFF_MERGE + 2 * SLOT;   // [2][8] float4 (m, m, l, l of rows i, i + 8), then [2] r
  static constexpr int OFF_BAR = OFF_STAT + 2 * 8 * 16 + 16;
  static constexpr int OFF_MISC = OFF_BAR + kWarps * STAGES * 8;
  static constexpr int OFF_NAN = OFF_MISC + 64;           // [D] first hidden key with a NaN value
  static constexpr int SMEM = OFF_NAN + 4 * D;
  static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two CTAs per SM");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ int pieces_of(const CacheParams& p, int b) {
  const int n = __ldg(p.cu_q + b + 1) - __ldg(p.cu_q + b);
  return n > 0 ? max(1, (__ldg(p.kv_lens + b) + kPiece - 1) / kPiece) : 0;
}

// Where a warp is in the CTA's run of pieces.
struct Cursor {
  int b, h;
  long long f, ubeg, uend;                   // piece, and the unit's first and last + 1
  __device__ __forceinline__ void settle(const CacheParams& p, long long end) {   // into the unit that holds f
    while (f < end && f >= uend) {
      ubeg = uend;
      if (++h == p.Hkv) {
        h = 0;
        int np;
        do np = pieces_of(p, ++b);           // f < end: there is another unit
        while (np == 0);
        uend = ubeg + np;
      } else {
        uend = ubeg + pieces_of(p, b);
      }
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    fwd_cache_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                            const CacheParams p, const int rows_max) {
  using C = DecCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = lane & 3, rq = lane >> 2;    // fragment column group and row
  long long* misc = reinterpret_cast<long long*>(smem + C::OFF_MISC);   // [4] warp sums / [0] b, [1] unit start
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 48);
  int* first_nan = reinterpret_cast<int*>(smem + C::OFF_NAN);
  int* any_nan = reinterpret_cast<int*>(smem + C::OFF_MISC + 52);
  const uint32_t bars = smem_u32(smem + C::OFF_BAR) + warp * C::STAGES * 8;
  const WaitCtl wc{p.wait_ns, p.status, abort_flag};
  const CacheWs W = cache_ws(gridDim.x, rows_max, D);
  char* ws = static_cast<char*>(p.ws);
  int4* rec = reinterpret_cast<int4*>(ws) + blockIdx.x;
  if (tid < D) first_nan[tid] = kNoKey;
  if (tid == 0) {
    *abort_flag = 0;
    *any_nan = 0;
    for (int i = 0; i < kWarps * C::STAGES; ++i) mbar_init(smem_u32(smem + C::OFF_BAR) + 8 * i, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }

  pdl_wait();                                // nothing of global memory before this
  pdl_trigger();
  // ---- the run of pieces of this CTA; thread t adds up sequences [t per_thread, ...)
  const int per_thread = (p.B + kThreads - 1) / kThreads;
  const int b_lo = min(tid * per_thread, p.B), b_hi = min(b_lo + per_thread, p.B);
  long long mine = 0;
  bool wrong = false;
  for (int b = b_lo; b < b_hi; ++b) {
    const int c0 = __ldg(p.cu_q + b), c1 = __ldg(p.cu_q + b + 1), len = __ldg(p.kv_lens + b), n = c1 - c0;
    wrong |= c0 < 0 || c1 < c0 || n > p.max_q || len < 0 || len > p.max_len || (p.causal && n > len) ||
             (b == 0 && c0 != 0) || (b == p.B - 1 && c1 != p.total_q);
    if (n > 0) mine += max(1, (len + kPiece - 1) / kPiece);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) misc[warp] = incl;
  const bool bad = __syncthreads_or(wrong) != 0;
  if (tid == 0) {
    *rec = make_int4(0, 0, 0, 0);            // no unit cut, unless found below
    if (bad) atomicExch(p.status, DEV_BAD_OFFSETS);
  }
  if (bad) return;
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += misc[w];
    total += misc[w];
  }
  total *= p.Hkv;
  before *= p.Hkv;
  mine *= p.Hkv;
  // Equal runs, but a piece for every warp at least: a shorter run would only add partial results.
  const long long run = max((total + gridDim.x - 1) / gridDim.x, (long long)kWarps);
  const long long rs = run * blockIdx.x, re = min(rs + run, total);
  if (rs >= total) return;
  __syncthreads();                           // misc has been read
  if (before <= rs && rs < before + mine) {
    int b = b_lo;
    long long at = before;
    for (;;) {
      const long long step = (long long)pieces_of(p, b) * p.Hkv;
      if (rs < at + step) break;
      at += step;
      ++b;
    }
    misc[0] = b;
    misc[1] = at;
  }
  __syncthreads();
  Cursor seg;                                // the unit being worked on
  seg.b = (int)misc[0];
  {
    const int np = pieces_of(p, seg.b);
    seg.h = (int)((rs - misc[1]) / np);
    seg.ubeg = misc[1] + (long long)seg.h * np;
    seg.uend = seg.ubeg + np;
    seg.f = rs;
  }

  // ---- this warp's loads, STAGES pieces ahead of its work
  const int page_shift = 31 - __clz(p.page);
  const int grp = lane & 1;                  // half of a piece (16 keys) this lane looks after
  uint8_t* ring = smem + warp * C::STAGES * 2 * C::KB;
  Cursor ahead = seg;
  ahead.f = rs + warp;
  ahead.settle(p, re);
  // The page of this lane's half of the piece at `ahead`: -1 behind the last key, -2 bad.
  auto page_at = [&]() -> int {
    if (ahead.f >= re) return -1;
    const int key = (int)(ahead.f - ahead.ubeg) * kPiece + grp * 16;
    if (key >= __ldg(p.kv_lens + ahead.b)) return -1;
    const int pg = __ldg(p.table + (long long)ahead.b * p.max_pages + (key >> page_shift));
    if (pg < 0 || pg >= p.num_pages) {
      atomicExch(p.status, DEV_BAD_PAGE);
      return -2;
    }
    return pg;
  };
  // Scale of this lane's half: K for lanes with bit 1 clear, V with it set.
  auto scale_of = [&](int pg, int h) -> float {
    return pg >= 0 ? __ldg(((lane & 2) ? p.v_scale : p.k_scale) + (long long)pg * p.Hkv + h) : 0.f;
  };
  auto issue = [&](int stage, int pg) {
    // Pages of 16 rows: two boxes, by lanes 0 and 1; larger ones hold the whole piece.
    const int p0 = __shfl_sync(0xffffffffu, pg, 0), p1 = __shfl_sync(0xffffffffu, pg, 1);
    const bool two = p.page == 16;
    const uint32_t bar = bars + 8 * stage;
    const uint32_t box = two ? C::KB / 2 : C::KB;
    if (lane == 0) {
      const int boxes = (p0 >= 0 ? 1 : 0) + (two && p1 >= 0 ? 1 : 0);
      mbar_arrive_expect_tx(bar, boxes * 2 * box);
    }
    __syncwarp();
    if (lane < (two ? 2 : 1) && pg >= 0) {
      const int key = (int)(ahead.f - ahead.ubeg) * kPiece + lane * 16;
      const int line = (key & (p.page - 1)) * D / 128;
      const int z = pg * p.Hkv + ahead.h;
      const uint32_t dst = smem_u32(ring + stage * 2 * C::KB) + lane * box;
      tma_load_3d(dst, &tm_k, 0, line, z, bar);
      tma_load_3d(dst + C::KB, &tm_v, 0, line, z, bar);
    }
  };
  int pages[C::STAGES + 1], heads[C::STAGES + 1];     // of the pieces under way, oldest first; one more looked up
  bool ok = true;
#pragma unroll
  for (int i = 0; i <= C::STAGES; ++i) {
    pages[i] = page_at();
    heads[i] = ahead.h;
    if (i < C::STAGES) {
      if (ahead.f < re && !(p.test_skip_first_kv && i == 0)) issue(i, pages[i]);
      ahead.f += kWarps;
      ahead.settle(p, re);
    }
  }
  // `ahead` now stands at piece number STAGES of this warp, whose page is pages[STAGES].
  float sc_next = scale_of(pages[0], heads[0]);
  int stage = 0;
  uint32_t phase = 0;
  long long f = rs + warp;                   // this warp's next piece

  // Shared-memory offsets of this thread's fragments within a piece.
  uint32_t koff[2], voff[2];
  if constexpr (D == 128) {
    const int kr = (rq & 1) ? (((rq - 1) ^ 4) + 1) : rq;          // row of fragment column rq: 0 5 2 7 4 1 6 3
    koff[0] = kr * 128 + ((c ^ kr) << 4);
    koff[1] = kr * 128 + (((c + 4) ^ kr) << 4);
    const int v0 = 2 * c, v1 = ((2 * c) ^ 4) + 1;
    voff[0] = v0 * 128 + ((rq ^ v0) << 4);
    voff[1] = v1 * 128 + ((rq ^ v1) << 4);
  } else {
    // Two rows of 64 bytes share a 128-byte line; within 16 rows fragment columns 2i, 2i+1 of the
    // first block are rows 4i, 4i+1 and of the second block rows 4i+2, 4i+3.
    const int line = (rq >> 1) * 2, half = rq & 1;
    koff[0] = line * 128 + (((half * 4 + c) ^ line) << 4);                    // first block
    koff[1] = (line + 1) * 128 + (((half * 4 + c) ^ (line + 1)) << 4);        // second block
    const int vl = 2 * c;
    voff[0] = vl * 128 + (((rq >> 1) ^ vl) << 4) + (rq & 1) * 8;              // first block, row 4c
    voff[1] = (vl + 1) * 128 + (((rq >> 1) ^ (vl + 1)) << 4) + (rq & 1) * 8;  // second block, row 4c + 2
  }

  const int g = p.g;
  // ---- units
  while (seg.f < re) {
    const int q0 = __ldg(p.cu_q + seg.b), n = __ldg(p.cu_q + seg.b + 1) - q0, len = __ldg(p.kv_lens + seg.b);
    const long long send = min(seg.uend, re);
    const int rows = n * g;
    // Visible keys of this thread's two rows.
    int lim[2];
    float crow[2];
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = rq + 8 * i, qi = r / g;
      lim[i] = p.causal && r < rows ? len - n + qi + 1 : len;
      uint4 w[D / 32];
      float amax = 0.f;
      const uint16_t* src = static_cast<const uint16_t*>(p.q) +
                            ((long long)(seg.h * g + (r - qi * g)) * p.total_q + q0 + qi) * D + c * 16;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {     // 16 columns at 16 c, and for d = 128 at 64 + 16 c
        w[k] = r < rows ? __ldg(reinterpret_cast<const uint4*>(src + (k >> 1) * 64) + (k & 1)) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          amax = fmax3(amax, fabsf(__uint_as_float(u[j] << 16)), fabsf(__uint_as_float(u[j] & 0xffff0000u)));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const uint32_t e = __float_as_uint(amax) >> 23;              // biased exponent
      const uint32_t up = min(268u - e, 253u);                     // of the factor: largest |q| to [2^14, 2^15)
      const float inv = __uint_as_float(up << 23);
      // A row that holds an infinity is NaN wherever it sees a key (as f16 it could be -inf at every key, which
      // would read as a row that sees none).
      crow[i] = p.c * (e < 255u ? __uint_as_float((254u - up) << 23) : __int_as_float(0x7fffffff));
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t h2 = pack_f16x2(__uint_as_float(u[j] << 16) * inv, __uint_as_float(u[j] & 0xffff0000u) * inv);
          // columns 16 c + 4 (step & 3) + {0, 1} are fragment columns 2c, 2c + 1, + {2, 3} are 2c + 8, 2c + 9
          const int word = (k & 1) * 4 + j;
          qf[(k >> 1) * 4 + (word >> 1)][(word & 1) * 2 + i] = h2;
        }
      }
    }
    const int min_lim = p.causal ? len - n + 1 : len;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, rref = kMinScale, rinv = 1.f / kMinScale;
    float o[C::NACC][4];
#pragma unroll
    for (int i = 0; i < C::NACC; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    // ---- this warp's pieces of the unit
    for (; f < send; f += kWarps) {
      const float sc = sc_next;
      const int key0 = (int)(f - seg.ubeg) * kPiece;
      const int pg = pages[0];
      if (ok && !__all_sync(0xffffffffu, mbar_wait(bars + 8 * stage, phase, wc))) {
        // A wait ran out: this warp loads and computes no more.  Its copies under way land first.
        ok = false;
        const unsigned long long t0 = globaltimer_ns();
        for (int k = 0; k < C::STAGES; ++k) {
          const int st = stage + k < C::STAGES ? stage + k : stage + k - C::STAGES;
          const uint32_t par = stage + k < C::STAGES ? phase : phase ^ 1u;
          if (f + (long long)k * kWarps < re)
            while (!mbar_try_wait(bars + 8 * st, par) && globaltimer_ns() - t0 < drain_ns(p)) {
            }
        }
        __syncwarp();
      }
      sc_next = scale_of(pages[1], heads[1]);
      if (ok) {
        const uint8_t* kt = ring + stage * 2 * C::KB;
        const uint8_t* vt = kt + C::KB;
        float s[4][4];
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
          if constexpr (D == 128) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint4 w = *reinterpret_cast<const uint4*>(kt + nb * 1024 + koff[k]);
              const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mma_f16(s[nb], qf[k * 4 + j][0], qf[k * 4 + j][1], qf[k * 4 + j][2], qf[k * 4 + j][3], e4m3x2_f16x2(u[j]),
                        e4m3x2_f16x2_hi(u[j]));
            }
          } else {
            const uint4 w = *reinterpret_cast<const uint4*>(kt + (nb >> 1) * 1024 + koff[nb & 1]);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_f16(s[nb], qf[j][0], qf[j][1], qf[j][2], qf[j][3], e4m3x2_f16x2(u[j]), e4m3x2_f16x2_hi(u[j]));
          }
        }
        const float ks[2] = {__shfl_sync(0xffffffffu, sc, 0), __shfl_sync(0xffffffffu, sc, 1)};
        const float vs[2] = {__shfl_sync(0xffffffffu, sc, 2), __shfl_sync(0xffffffffu, sc, 3)};
        const bool got0 = __shfl_sync(0xffffffffu, pg, 0) >= 0, got1 = __shfl_sync(0xffffffffu, pg, 1) >= 0;
        const bool partial = key0 + kPiece > min_lim || !got0 || !got1;
        // Key of fragment column 2c + e of block nb, relative to the piece.
        auto key_of = [&](int nb, int e) -> int {
          if constexpr (D == 128) return nb * 8 + (e ? ((2 * c) ^ 4) + 1 : 2 * c);
          else return (nb >> 1) * 16 + 4 * c + 2 * (nb & 1) + e;
        };
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[nb][i] *= ks[nb >> 1] * crow[i >> 1];
        if (partial) {
          // V of a key that some queries do not see (its row: D / 16 pieces, for d = 64 half a line).
          const int key = key0 + lane;
          if (key >= min_lim && key < len && (lane < 16 ? got0 : got1)) {
            const int line = D == 128 ? lane : lane >> 1, at = D == 128 ? 0 : (lane & 1) * 4;
            uint8_t* row = ring + stage * 2 * C::KB + C::KB + line * 128;
#pragma unroll 1
            for (int x = 0; x < D / 16; ++x) {
              uint8_t* piece = row + (((at + x) ^ (line & 7)) << 4);
              if (any_nan_code(*reinterpret_cast<const uint4*>(piece))) {
                take_nan_codes(piece, key, first_nan + x * 16, any_nan);
                fence_proxy_async_smem();    // a copy into this stage comes next
              }
            }
          }
          __syncwarp();
#pragma unroll
          for (int nb = 0; nb < 4; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (key0 + key_of(nb, i & 1) >= lim[i >> 1] || !((nb >> 1) ? got1 : got0)) s[nb][i] = -INFINITY;
        }
        float mx[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float a = fmax3(s[0][2 * i], s[0][2 * i + 1], s[1][2 * i]);
          a = fmax3(a, s[1][2 * i + 1], s[2][2 * i]);
          a = fmax3(a, s[2][2 * i + 1], s[3][2 * i]);
          a = fmaxf(a, s[3][2 * i + 1]);
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
          mx[i] = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
        }
        const float vmax = fmaxf(vs[0], vs[1]);
        if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1]) || vmax > rref) {
          float fac = 1.f;
          if (vmax > rref) {
            rinv = 1.f / vmax;
            fac = rref * rinv;
            rref = vmax;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float mn = fmaxf(m[i], mx[i]);
            const float alpha = mn == -INFINITY ? 1.f : ex2_mufu(m[i] - mn);
            m[i] = mn;
            l[i] *= alpha;
#pragma unroll
            for (int j = 0; j < C::NACC; ++j) {
              o[j][2 * i] *= alpha * fac;
              o[j][2 * i + 1] *= alpha * fac;
            }
          }
        }
        uint32_t pf[4][2];
        const float vw[2] = {vs[0] * rinv, vs[1] * rinv};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float off = kShift - (m[i] == -INFINITY ? 0.f : m[i]);
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) {
            const float a = ex2_mufu(s[nb][2 * i] + off), b = ex2_mufu(s[nb][2 * i + 1] + off);
            l[i] += a + b;
            pf[nb][i] = pack_f16x2(a * vw[nb >> 1], b * vw[nb >> 1]);
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          // Rows of V behind the last key may hold any code (NaN too): their weight is 0, their value must be.
          bool live[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            live[x] = key0 + key_of(2 * t + (x >> 1), x & 1) < len && (t ? got1 : got0);
          if constexpr (D == 128) {
            uint4 v[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              v[x] = *reinterpret_cast<const uint4*>(vt + t * 2048 + (x >> 1) * 1024 + voff[x & 1]);
              if (partial && !live[x]) v[x] = make_uint4(0u, 0u, 0u, 0u);
            }
            const uint32_t u[4][4] = {{v[0].x, v[0].y, v[0].z, v[0].w}, {v[1].x, v[1].y, v[1].z, v[1].w},
                                      {v[2].x, v[2].y, v[2].z, v[2].w}, {v[3].x, v[3].y, v[3].z, v[3].w}};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t a = __byte_perm(u[0][w], u[1][w], 0x5140), b = __byte_perm(u[0][w], u[1][w], 0x7362);
              const uint32_t e = __byte_perm(u[2][w], u[3][w], 0x5140), d = __byte_perm(u[2][w], u[3][w], 0x7362);
              mma_f16(o[4 * w], pf[2 * t][0], pf[2 * t][1], pf[2 * t + 1][0], pf[2 * t + 1][1], e4m3x2_f16x2(a), e4m3x2_f16x2(e));
              mma_f16(o[4 * w + 1], pf[2 * t][0], pf[2 * t][1], pf[2 * t + 1][0], pf[2 * t + 1][1], e4m3x2_f16x2_hi(a), e4m3x2_f16x2_hi(e));
              mma_f16(o[4 * w + 2], pf[2 * t][0], pf[2 * t][1], pf[2 * t + 1][0], pf[2 * t + 1][1], e4m3x2_f16x2(b), e4m3x2_f16x2(d));
              mma_f16(o[4 * w + 3], pf[2 * t][0], pf[2 * t][1], pf[2 * t + 1][0], pf[2 * t + 1][1], e4m3x2_f16x2_hi(b), e4m3x2_f16x2_hi(d));
            }
          } else {
            // Rows 4c and 4c + 1 (first block) are the halves of one line, as are 4c + 2, 4c + 3.
            uint2 v[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              v[x] = *reinterpret_cast<const uint2*>(vt + t * 1024 + (voff[x >> 1] ^ ((x & 1) << 6)));
              if (partial && !live[x]) v[x] = make_uint2(0u, 0u);
            }
            const uint32_t u[4][2] = {{v[0].x, v[0].y}, {v[1].x, v[1].y}, {v[2].x, v[2].y}, {v[3].x, v[3].y}};
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const uint32_t a = __byte_perm(u[0][w], u[1][w], 0x5140), b = __byte_perm(u[0][w], u[1][w], 0x7362);
              const uint32_t e = __byte_perm(u[2][w], u[3][w], 0x5140), d = __byte_perm(u[2][w], u[3][w], 0x7362);
              mma_f16(o[4 * w], pf[2 * t][0], pf[2 * t][1], pf[2 * t + 1][0], pf[2 * t + 1][1], e4m3x2_f16x2(a), e4m3x2_f16x2(e));
              mma_f16(o[4 * w + 1], pf[2 * t][0], pf[2 * t][1], pf[2 * t + 1][0], pf[2 * t + 1][1], e4m3x2_f16x2_hi(a), e4m3x2_f16x2_hi(e));
              mma_f16(o[4 * w + 2], pf[2 * t][0], pf[2 * t][1], pf[2 * t + 1][0], pf[2 * t + 1][1], e4m3x2_f16x2(b), e4m3x2_f16x2(d));
              mma_f16(o[4 * w + 3], pf[2 * t][0], pf[2 * t][1], pf[2 * t + 1][0], pf[2 * t + 1][1], e4m3x2_f16x2_hi(b), e4m3x2_f16x2_hi(d));
            }
          }
        }
      }
      // The stage is read: the next piece into it.
      __syncwarp();
      if (ok && ahead.f < re) issue(stage, pages[C::STAGES]);
#pragma unroll
      for (int i = 0; i < C::STAGES; ++i) {
        pages[i] = pages[i + 1];
        heads[i] = heads[i + 1];
      }
      ahead.f += kWarps;
      ahead.settle(p, re);
      pages[C::STAGES] = page_at();
      heads[C::STAGES] = ahead.h;
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }

    // ---- the four warps' results of the unit into one (warp 0)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    float4* slots = reinterpret_cast<float4*>(smem + C::OFF_MERGE);
    float4* stats = reinterpret_cast<float4*>(smem + C::OFF_STAT);
    float* refs = reinterpret_cast<float*>(smem + C::OFF_STAT + 2 * 8 * 16);
    auto put = [&](int slot) {
#pragma unroll
      for (int j = 0; j < C::NACC; ++j) slots[(slot * C::NACC + j) * 32 + lane] = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
      if (c == 0) stats[slot * 8 + rq] = make_float4(m[0], m[1], l[0], l[1]);
      if (lane == 0) refs[slot] = rref;
    };
    auto take = [&](int slot) {
      const float4 st = stats[slot * 8 + rq];
      const float ro = refs[slot], rn = fmaxf(rref, ro), ri = 1.f / rn;
      const float mo[2] = {st.x, st.y}, lo[2] = {st.z, st.w};
      float wa[2], wb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mn = fmaxf(m[i], mo[i]), mu = mn == -INFINITY ? 0.f : mn;
        wa[i] = ex2_mufu(m[i] - mu);
        wb[i] = ex2_mufu(mo[i] - mu);
        l[i] = l[i] * wa[i] + lo[i] * wb[i];
        m[i] = mn;
        wa[i] *= rref * ri;
        wb[i] *= ro * ri;
      }
      rref = rn;
#pragma unroll
      for (int j = 0; j < C::NACC; ++j) {
        const float4 x = slots[(slot * C::NACC + j) * 32 + lane];
        o[j][0] = o[j][0] * wa[0] + x.x * wb[0];
        o[j][1] = o[j][1] * wa[0] + x.y * wb[0];
        o[j][2] = o[j][2] * wa[1] + x.z * wb[1];
        o[j][3] = o[j][3] * wa[1] + x.w * wb[1];
      }
    };
    __syncthreads();                         // the slots are free
    const bool nan = *any_nan != 0;
    if (nan && warp == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i)            // o[j][i]: row i / 2, column see below
#pragma unroll
        for (int j = 0; j < C::NACC; ++j)
          if (first_nan[c * (D / 4) + (i & 1) * (D / 8) + j] < lim[i >> 1]) o[j][i] = __int_as_float(0x7fffffff);
    }
    if (warp >= 2) put(warp - 2);
    __syncthreads();
    if (warp < 2) take(warp);
    if (warp == 1) {                         // only warp 1 reads this slot; its lanes share the statistics, so all
      __syncwarp();                          // of them have read before some write
      put(1);
    }
    if (nan && warp == 3) {
      for (int i = lane; i < D; i += 32) first_nan[i] = kNoKey;
      if (lane == 0) *any_nan = 0;
    }
    __syncthreads();
    if (warp == 0) {
      take(1);
      const bool whole = seg.ubeg >= rs && seg.uend <= re;
      // First unit of the CTA: partial 0, its last one: partial 1.
      const int second = seg.ubeg > rs ? 1 : 0, part = 2 * blockIdx.x + second;
      if (seg.ubeg >= rs && !whole && lane == 0)
        *rec = make_int4(seg.h, q0, n, 2 * ((int)((seg.uend - 1) / run) - (int)blockIdx.x) + second);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = rq + 8 * i, qi = r / g;
        if (r >= rows) continue;
        // Columns of o[j][2i] and o[j][2i + 1]: for d = 128, 32 c + j and 32 c + 16 + j; d = 64, 16 c + j and 16 c + 8 + j.
        if (whole) {
          const float inv = l[i] == 0.f ? 0.f : rref / l[i];
          const long long row = (long long)(seg.h * g + (r - qi * g)) * p.total_q + q0 + qi;
          uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + row * D + c * (D / 4));
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int k = 0; k < C::NACC / 8; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                w[x] = pack_bf16x2(o[8 * k + 2 * x][2 * i + e] * inv, o[8 * k + 2 * x + 1][2 * i + e] * inv);
              out[e * (C::NACC / 8) + k] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          if (c == 0) p.lse[row] = (m[i] - kShift + __log2f(l[i])) * kLn2;
        } else {
          float4* out = reinterpret_cast<float4*>(ws + W.part) + ((long long)part * (D / 4) + c * (D / 16)) * rows_max + r;
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int k = 0; k < C::NACC / 4; ++k)
              out[(e * (C::NACC / 4) + k) * rows_max] = make_float4(o[4 * k][2 * i + e], o[4 * k + 1][2 * i + e], o[4 * k + 2][2 * i + e],
                                                       o[4 * k + 3][2 * i + e]);
          if (c == 0)
            reinterpret_cast<float4*>(ws + W.stat)[(long long)part * rows_max + r] = make_float4(m[i] - kShift, l[i], rref, 0.f);
        }
      }
    }
    seg.f = send;
    seg.settle(p, re);
  }
}

// Joins the partial results of cut units.  An item is 128 threads' share of a unit that starts in one
// CTA of the main kernel and goes on in others (at most one per CTA): a thread has one row and CPT
// neighbouring pieces of 4 columns of it, and reads JOIN partials' statistics and pieces at once, joining
// them as they come.  CPT = JOIN = 2 when there are many units (bytes and the blocks in flight bound it:
// of two prompts of 4096, 152 units of 256 rows, 11 us of 680; CPT = JOIN = 4 took 2 us longer), CPT = 1
// and JOIN = 8 for decoding and for few units (latency does; JOIN = 4 or 16 is slower).
// COMPACT: the blocks first look which CTAs left a unit and share these units' items; otherwise block i
// takes item i of all CTAs, which is one look-up shorter but comes to several waves of blocks that find
// nothing when few CTAs leave a unit of many items (4 drafted tokens, 8 units: 25.1 us against 26.1;
// 16 sequences of 16 rows in 1216 blocks 99.6 against 97.6, with many units 3 us more).
template <int D, int CPT, int JOIN, bool COMPACT>
__global__ void __launch_bounds__(128) fwd_cache_merge_kernel(const CacheParams p, const int rows_max, const int row_shift,
                                                              const int ctas) {
  constexpr int GROUPS = D / 4 / CPT;
  static_assert(CPT <= 2, "one store per row and thread");
  __shared__ uint32_t cut[32];               // bit i: CTA i left a unit (COMPACT: at most 1024 CTAs)
  const CacheWs W = cache_ws(ctas, rows_max, D);
  const char* ws = static_cast<const char*>(p.ws);
  const int4* recs = reinterpret_cast<const int4*>(ws);
  pdl_wait();
  pdl_trigger();
  int units = ctas;
  if constexpr (COMPACT) {
    for (int i = threadIdx.x; i < (ctas + 31) / 32 * 32; i += 128) {
      const uint32_t b = __ballot_sync(0xffffffffu, i < ctas && recs[min(i, ctas - 1)].w >= 2);
      if ((i & 31) == 0) cut[i >> 5] = b;
    }
    __syncthreads();
    units = 0;
    for (int i = 0; i < (ctas + 31) / 32; ++i) units += __popc(cut[i]);
  }
  const int shares = ((GROUPS << row_shift) + 127) / 128;
  for (int item = blockIdx.x; item < units * shares; item += gridDim.x) {
    const int share = item / units;
    int cta = item - share * units;
    if constexpr (COMPACT) {                 // the cta-th bit set
      int w = 0;
      while (cta >= __popc(cut[w])) cta -= __popc(cut[w++]);
      uint32_t bits = cut[w];
      for (; cta > 0; --cta) bits &= bits - 1;
      cta = w * 32 + __ffs(bits) - 1;
    }
    const int t = share * 128 + threadIdx.x, r = t & ((1 << row_shift) - 1), cg = t >> row_shift;
    const int qi = r / p.g;
    const float4* stat = reinterpret_cast<const float4*>(ws + W.stat) + r;
    const float4* part = reinterpret_cast<const float4*>(ws + W.part) + (long long)cg * CPT * rows_max + r;
    const int4 rec = recs[cta];
    if (rec.w < 2 || qi >= rec.z || cg >= GROUPS) continue;
    const int first = 2 * cta + (rec.w & 1), more = rec.w >> 1;
    // The unit's partials: the first CTA's, then partial 0 of each CTA behind it.
    auto which = [&](int k) -> long long { return k == 0 ? first : 2 * (cta + k); };
    float m = -INFINITY, ref = kMinScale, l = 0.f;
    float4 o[CPT];
#pragma unroll
    for (int c = 0; c < CPT; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 <= more; k0 += JOIN) {
      float4 x[JOIN][CPT], st[JOIN];
#pragma unroll
      for (int j = 0; j < JOIN; ++j) {
        const long long w = which(min(k0 + j, more));     // (the last one again: loads without conditions)
        st[j] = stat[w * rows_max];
#pragma unroll
        for (int c = 0; c < CPT; ++c) x[j][c] = part[(w * (D / 4) + c) * rows_max];
      }
      float mn = m, rn = ref;
#pragma unroll
      for (int j = 0; j < JOIN; ++j) {
        mn = fmaxf(mn, st[j].x);
        rn = fmaxf(rn, st[j].z);
      }
      const float mu = mn == -INFINITY ? 0.f : mn, rinv = 1.f / rn;
      const float w0 = ex2_mufu(m - mu), v0 = w0 * (ref * rinv);
      l *= w0;
#pragma unroll
      for (int c = 0; c < CPT; ++c) { o[c].x *= v0; o[c].y *= v0; o[c].z *= v0; o[c].w *= v0; }
#pragma unroll
      for (int j = 0; j < JOIN; ++j) {
        if (k0 + j > more) break;
        const float w = ex2_mufu(st[j].x - mu), v = w * (st[j].z * rinv);
        l += w * st[j].y;
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
          o[c].x += v * x[j][c].x;
          o[c].y += v * x[j][c].y;
          o[c].z += v * x[j][c].z;
          o[c].w += v * x[j][c].w;
        }
      }
      m = mn;
      ref = rn;
    }
    const long long row = (long long)(rec.x * p.g + r - qi * p.g) * p.total_q + rec.y + qi;
    const float inv = l == 0.f ? 0.f : ref / l;
    uint32_t y[2 * CPT];
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      y[2 * c] = pack_bf16x2(o[c].x * inv, o[c].y * inv);
      y[2 * c + 1] = pack_bf16x2(o[c].z * inv, o[c].w * inv);
    }
    uint16_t* out = static_cast<uint16_t*>(p.o) + row * D + cg * CPT * 4;
    if constexpr (CPT == 1) *reinterpret_cast<uint2*>(out) = make_uint2(y[0], y[1]);
    else *reinterpret_cast<uint4*>(out) = make_uint4(y[0], y[1], y[2], y[3]);
    if (cg == 0) p.lse[row] = (m + __log2f(l)) * kLn2;
  }
}

template <int D>
cudaError_t launch_decode(const CacheMaps& maps, const CacheParams& p, int rows, int grid, cudaStream_t s) {
  using C = DecCfg<D>;
  static std::once_flag flags[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::call_once(flags[dev & 63], [&] {
    attr_err[dev & 63] = cudaFuncSetAttribute(fwd_cache_decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (attr_err[dev & 63] != cudaSuccess) return attr_err[dev & 63];
  // A dependent launch of whatever runs before: the kernel waits for it to be done, but is in place by then.
  e = launch_pdl(fwd_cache_decode_kernel<D>, dim3(grid), dim3(kThreads), C::SMEM, s, maps.k, maps.v, p, rows);
  if (e != cudaSuccess) return e;
  return launch_fwd_cache_merge(p, D, rows, grid, s);
}

}  // namespace

cudaError_t launch_fwd_cache_merge(const CacheParams& p, int d, int rows, int ctas, cudaStream_t s) {
  int shift = 0;
  while ((1 << shift) < rows && (1 << shift) < (long long)p.max_q * p.g) ++shift;     // rows in use
  auto go = [&](auto kernel, int cpt, bool compact) {
    const int shares = (((d / 4 / cpt) << shift) + 127) / 128;
    const int blocks = compact ? 4 * kSMs : ctas * shares;
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(128), 0, s, p, rows, shift, ctas);
  };
  // Few units of many partials each: latency again (a sequence of 30000 keys, 32 rows: 33 us against 35).
  const long long units = (long long)p.B * p.Hkv * (((long long)p.max_q * p.g + rows - 1) / rows);
  if (rows <= kCacheDecodeRows || units * 4 <= ctas) {
    if (((d / 4) << shift) / 128 * ctas > 16 * kSMs && ctas <= 1024)
      return d == 64 ? go(fwd_cache_merge_kernel<64, 1, 8, true>, 1, true) : go(fwd_cache_merge_kernel<128, 1, 8, true>, 1, true);
    return d == 64 ? go(fwd_cache_merge_kernel<64, 1, 8, false>, 1, false) : go(fwd_cache_merge_kernel<128, 1, 8, false>, 1, false);
  }
  return d == 64 ? go(fwd_cache_merge_kernel<64, 2, 2, false>, 2, false) : go(fwd_cache_merge_kernel<128, 2, 2, false>, 2, false);
}

size_t cache_decode_workspace_bytes(int rows, int d, int sms) { return cache_ws(2 * sms, rows, d).total; }

cudaError_t launch_fwd_cache_decode(const CacheMaps& maps, const CacheParams& p, int d, int sms, cudaStream_t s) {
  const int rows = p.max_q * p.g, grid = 2 * sms;      // as in the workspace's size
  return d == 64 ? launch_decode<64>(maps, p, rows, grid, s) : launch_decode<128>(maps, p, rows, grid, s);
}

}  // namespace attn
