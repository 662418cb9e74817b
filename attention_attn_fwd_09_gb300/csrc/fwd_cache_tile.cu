// Attention of packed queries over a paged e4m3 cache: many query rows per K/V head (pieces of
// prompts, drafts).  fwd_cache.cu is the kernel for up to 16 rows.
//
// A unit is up to 256 rows of one sequence and K/V head as two 128-row tiles: row r is query r / g,
// head r % g of the group, so every tile is full whatever g is and the g heads share the K, V
// they share.  What bounds it is the tensor cores and, behind them, each tile's own chain S ->
// softmax -> P -> PV, so two tiles run half a turn apart and one's products cover the other's
// softmax.  16 warps, a persistent CTA per SM:
//   * producer: K, V codes by TMA, a box per page;
//   * two MMA issuers, one per tile, that take turns (one thread for both lost 1000 cycles per block
//     in its waits; two without turns fall into step).  A group of products is PV of one block and S
//     of the next; its completion frees the slots that it read;
//   * scheduler: walks the CTA's units and describes each in shared memory, up to four ahead;
//   * two softmax warpgroups, a row per thread.  They prepare Q, rescale O themselves when a maximum
//     grew by more than tau or a larger V scale came (rare after the first blocks), and hand P over
//     in two halves, so that PV begins before the second half's exponentials;
//   * a warpgroup that widens V and writes the results.
// Numbers:
//   * S on the 8-bit tensor path, K's codes as they lie in the cache.  Q, scaled by a power of two
//     per row (largest |q| in [128, 256)), is the sum of two 8-bit tiles, Q1 = e4m3(q) and
//     Q2 = e5m2(q - Q1).  bf16 has 8 significant bits and e4m3 4, so what Q1 leaves of a component
//     with exponent e >= -6 is 0 to 8 times 2^(e - 7): at most 3 significant bits and not below
//     2^-13, which e5m2 holds (e4m3, whose step ends at 2^-9, does so from e = -2 on).  The sum is
//     q itself down to 2^-13 of the row's largest component; below that Q1 leaves at most 2^-10, of
//     which e5m2 misses at most 2^-14: 2^-21 of the row's largest (e4m3: all of it, 2^-17).
//     Both products together cost what one 16-bit product costs, and K needs no widening;
//   * V widened to f16, times its page's scale over the largest V scale so far, times 2^7 (448 * 2^7
//     < 65504): a page's codes keep their bits down to 2^-17 of the largest scale.  Weights are held
//     times 2^7 (2^8 at most times tau's 2^8) in f16.
// The work is cut evenly: all units' 128-key blocks laid end to end, with a cost for starting and
// ending a unit, and every CTA takes an equal run.  Units cut between CTAs leave partial results for
// the merge kernel.
//
// SPLIT (no sequence has more than 128 rows per K/V head): both tiles hold the same rows and take
// the unit's blocks in turn, joined in tensor memory at the end.  With one tile idle a block took
// its whole chain, 3850 cycles; taken in turn 2100.  One Q instead of two leaves room for four K slots.
//
// Measured: two prompts of 4096 over 8192 keys, 32 heads on 8, d = 128: 680 us, 1212 TFLOP/s (a
// two-tile step of 128 keys takes 3900 cycles, of which the tensor cores need 2050 and shared memory
// 2180); four pieces of up to 512 over up to 16000 keys: 234 us, 1093 TFLOP/s.  SPLIT: 16 sequences
// of 16000 keys, 8 K/V heads of 32 rows: 141 us, 3.7 TB/s of cache (198 us without).  d = 64, where a
// key's exponentials cost the same for half the products: the prompts 577 us, 715 TFLOP/s.  Keys in two
// parts: 24 pieces of up to 60 queries behind prefixes of 5000, 0 and 16001 keys, 16 heads on 2, d = 64, 66 us;
// one prefix of 32768 keys, all rows of 64 sequences' 32 heads on 8, 48 us, 21000 of its 90000 cycles before
// the first scores and 12000 on the results.
//
// Shared memory (d = 128): Q1, Q2 2 x 32 KB, K8 ring 2 x 16 KB, V8 ring 3 x 16 KB, V16 2 x 32 KB.
// TMEM: S0 [0,128) S1 [128,256) O0 [256,384) O1 [384,512); P_t (f16 pairs) overwrites S_t.
#ifndef CACHE_TILE_SIDE
#define CACHE_TILE_SIDE false                // fwd_cache_tile_side.cu: this file again, keys in two parts
#endif
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "cache.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kTThreads = 512;
constexpr int kTRows = 256;                  // rows of a unit
constexpr float kPShift = 7.f;               // weights are held times 2^7
constexpr float kVShift = 128.f;             // and V times 2^7 over the reference scale
constexpr float kTau = 8.f;                  // rescale when a maximum grows by more (2^(7 + 8) < 65504)
constexpr int kUnitCost = 5;                 // at most what starting and ending a unit counts for, in key blocks
constexpr float kMinFactor = 1e-30f;         // keeps -inf * factor = -inf for pages whose scale is 0

template <int D, bool SPLIT>
struct TileCfg {
  static constexpr uint32_t Q8 = 128 * D;          // one 8-bit tile of Q
  static constexpr uint32_t K8 = 128 * D;          // 128 keys of e4m3 K or V
  static constexpr uint32_t CH16 = 128 * 128;      // 128 keys x 64 f16 columns (a swizzled box)
  static constexpr uint32_t V16 = (D / 64) * CH16;
  static constexpr int NK = SPLIT ? 4 : 2, NV8 = 3, NV16 = 2;   // ring slots
  static constexpr uint32_t OFF_Q = 0;             // [tile][Q1, Q2] (SPLIT: one tile's)
  static constexpr uint32_t OFF_K = OFF_Q + (SPLIT ? 2 : 4) * Q8;
  static constexpr int RELS = SPLIT ? 16 : 8;      // release barriers: more than the groups that K's ring spans
  static constexpr uint32_t OFF_V8 = OFF_K + NK * K8;
  static constexpr uint32_t OFF_V16 = OFF_V8 + NV8 * K8;
  static constexpr uint32_t OFF_CTRL = OFF_V16 + NV16 * V16;
  static constexpr uint32_t CTRL_BYTES = 512 + 256 + 6 * 128 * 4 + 64 + 2 * D * 4;
  static constexpr uint32_t SMEM = 1024 + OFF_CTRL + CTRL_BYTES;
  // K-major rows of D bytes: 128-byte swizzle for d = 128, 64-byte for d = 64.
  static constexpr uint32_t IDESC_Q1K = idesc_f32acc(128, 128, FMT_E4M3, FMT_E4M3, false, false);
  static constexpr uint32_t IDESC_Q2K = idesc_f32acc(128, 128, FMT_E5M2, FMT_E4M3, false, false);
  static constexpr uint32_t IDESC_PV = idesc_f32acc(128, D, FMT_F16, FMT_F16, false, true);
  static constexpr uint32_t QK_HI = D == 128 ? sdesc_sw128_hi(1024) : ((512u >> 4) | (1u << 14) | (4u << 29));
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

enum {
  T_Q = 0,         // +t: Q_t of the unit written (128)
  T_SFULL = 2,     // +t: S_t of a block complete
  T_PFULL = 4,     // +t: P written (128)
  T_OFULL = 6,     // +t: the unit's last PV of tile t complete
  T_OFREE = 8,     // +t: O_t read out of tensor memory (128)
  T_FIN = 10,      // +t: the unit's final statistics written (128)
  T_KFULL = 12,    // +slot (up to 4)
  T_V8FULL = 16,   // +slot (3)
  T_V8FREE = 19,   // +slot (3): widened (128)
  T_V16FULL = 22,  // +slot (2): widened (128)
  T_EPI = 24,      // the unit's results written (128)
  T_UFULL = 25,    // +slot (4): unit descriptor written
  T_UFREE = 29,    // +slot (4): every role is through with the unit (15 warps)
  T_DONE = 33,     // +t
  T_TURN = 35,     // +t: the other tile's products of a group have been issued
  T_PHALF = 37,    // +t: P of the block's first 64 keys written and O rescaled (128)
  T_REL = 39,      // +(group mod 8 or 16): both issuers' products of the group complete
  T_COUNT = 55
};
static_assert(T_COUNT * 8 <= 512, "barriers fit the control block's first 512 bytes");
constexpr int kUnitSlots = 4, kUnitReaders = 15;   // producer, 2 MMA issuers, 8 softmax and 4 widening warps

// sum_{i=0}^{n-1} floor((a i + b) / m), for a n + b < 2^32 (64-bit divisions made a CTA's start 4 us
// longer).  The sum counts lattice points under a line; taking whole parts of a / m and b / m out and
// then exchanging the axes turns (a, m) into (m, a mod m), as Euclid's algorithm does, so it ends after
// O(log) steps.
__device__ __forceinline__ long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  long long s = 0;
  while (n > 0) {
    s += (long long)(n - 1) * n / 2 * (a / m) + (long long)n * (b / m);
    a %= m;
    b %= m;
    const uint32_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return s;
}

// A sequence: its units per K/V head and their blocks of 128 keys.  Unit rt holds queries rt qu ..
// rt qu + qu - 1, qu = 256 / g.  Work is counted in steps: a unit's blocks and `cost` steps before
// them (CTAs with many short units took 1.4 times as long when blocks alone were counted).
// SIDE: sequences of either part.
template <bool SIDE>
struct TileSeq {
  int q0, n, len, units, causal;
  __device__ __forceinline__ TileSeq(const CacheParams& p, int b, int qu) {
    if constexpr (SIDE) {
      const PartSeq s(p, b);
      q0 = __ldg(s.cu + s.b);
      n = __ldg(s.cu + s.b + 1) - q0;
      len = __ldg(s.lens + s.b);
      causal = s.causal;
    } else {
      q0 = __ldg(p.cu_q + b);
      n = __ldg(p.cu_q + b + 1) - q0;
      len = __ldg(p.kv_lens + b);
      causal = p.causal;
    }
    units = (int)(((unsigned)max(n, 0) + qu - 1) / qu);
  }
  __device__ __forceinline__ int blocks(const CacheParams& p, int qu, int rt) const {
    const int lim = causal ? len - n + min(n, (rt + 1) * qu) : len;
    return (max(lim, 1) + 127) / 128;
  }
  // Blocks of the units before rt (a unit without keys counts as one).
  __device__ __forceinline__ long long blocks_before(const CacheParams& p, int qu, int rt) const {
    if (rt <= 0) return 0;
    if (!causal) return (long long)rt * ((max(len, 1) + 127) / 128);
    if (rt < units) return floor_sum(rt, 128, qu, (uint32_t)(len - n) + qu + 127);
    return floor_sum(units - 1, 128, qu, (uint32_t)(len - n) + qu + 127) + (len + 127) / 128;
  }
};

// A unit as the roles see it (shared memory, written by the scheduler warp).
struct __align__(16) UnitDesc {
  int nmax;                                  // key blocks here: of the longer tile (-1: no more units)
  int nt[2];                                 // and of each tile (SPLIT: its share of them)
  int kt0;                                   // first key block here
  int len;                                   // the sequence's keys
  int b, h;
  int rows;                                  // in use of 256
  int q0;                                    // first packed query
  int lim0;                                  // visible keys of the first query (not causal: of all)
  int whole;                                 // the unit is this CTA's alone
  int second;                                // partial 1 of the CTA, else partial 0
  int more;                                  // CTAs behind this one that go on with it, if it starts here (else -1)
  int causal, part, pad;                     // SIDE: of the sequence's part
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtl& w) {
  const bool ok = mbar_wait(bar, parity, w);
  return __all_sync(0xffffffffu, ok);
}
template <int N>
__device__ __forceinline__ void reg_fence(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i])::"memory");
}

// Two fp32 values -> two e4m3 or e5m2 codes (low byte: a).
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ uint32_t to_e5m2x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// 32 lanes x 16 consecutive 32-bit columns of tensor memory.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// NG: groups of columns of a key block that may have scales of their own, one per page of it.
// SIDE: keys in two parts (p.side); a template, since its registers would spill in the ordinary epilogue.
template <int D, int NG, bool SPLIT, bool SIDE>
__global__ void __launch_bounds__(kTThreads, 1)
    fwd_cache_tile_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                          const CacheParams p) {
  constexpr int KG = 128 / NG;               // keys of a group
  using C = TileCfg<D, SPLIT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint8_t* ctrl = smem + C::OFF_CTRL;
  const uint32_t bar0 = smem_u32(ctrl);
  auto BAR = [&](int i) -> uint32_t { return bar0 + 8u * i; };
  UnitDesc* desc = reinterpret_cast<UnitDesc*>(ctrl + 512);  // [4]
  float* fin = reinterpret_cast<float*>(ctrl + 768);         // [2][m, l, reference scale][128]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(fin + 768);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  long long* misc = reinterpret_cast<long long*>(tmem_slot + 2);   // [4]: b, h, rt, unit start
  int* any_nan = reinterpret_cast<int*>(misc + 4);                 // [2] by the unit's parity
  int* nan_keys = reinterpret_cast<int*>(tmem_slot + 16);          // [2][D] first hidden key with a NaN value
  long long* sums = reinterpret_cast<long long*>(smem + C::OFF_Q); // [16][2] warp sums, before Q is written

  const int tid = threadIdx.x, warp = warp_id(), lane = lane_id(), wg = warp >> 2;
  const int qu = kTRows / p.g;                               // queries per unit
  constexpr int LAG = SPLIT ? 2 : 1;                         // groups from a block's S to its PV
  const WaitCtl wc{p.wait_ns, p.status, abort_flag};
  const CacheWs W = cache_ws(gridDim.x, kTRows, D);
  char* ws = static_cast<char*>(p.ws);
  int4* rec = reinterpret_cast<int4*>(ws) + blockIdx.x;

  if (tid < 2 * D) nan_keys[tid] = kNoKey;
  if (tid == 0) {
    mbar_init(BAR(T_EPI), 128);
    for (int i = 0; i < kUnitSlots; ++i) {
      mbar_init(BAR(T_UFULL + i), 1);
      mbar_init(BAR(T_UFREE + i), kUnitReaders);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(BAR(T_Q + t), 128);
      mbar_init(BAR(T_SFULL + t), 1);
      mbar_init(BAR(T_PFULL + t), 128);
      mbar_init(BAR(T_PHALF + t), 128);
      mbar_init(BAR(T_V16FULL + t), 128);
      mbar_init(BAR(T_OFULL + t), 1);
      mbar_init(BAR(T_OFREE + t), 128);
      mbar_init(BAR(T_FIN + t), 128);
      mbar_init(BAR(T_DONE + t), 1);
      mbar_init(BAR(T_TURN + t), 1);
    }
    for (int s = 0; s < C::NV8; ++s) {
      mbar_init(BAR(T_V8FULL + s), 1);
      mbar_init(BAR(T_V8FREE + s), 128);
    }
    for (int i = 0; i < C::NK; ++i) mbar_init(BAR(T_KFULL + i), 1);
    for (int i = 0; i < C::RELS; ++i) mbar_init(BAR(T_REL + i), SPLIT ? 1 : 2);
    *abort_flag = 0;
    any_nan[0] = any_nan[1] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }

  pdl_wait();                                // nothing of global memory before this
  pdl_trigger();
  // ---- the run of steps of this CTA; thread t adds up sequences [t per_thread, ...)
  const int seqs = SIDE && p.side == SIDE_BOTH ? p.B + p.two.B : p.B;
  const int per_thread = (seqs + kTThreads - 1) / kTThreads;
  const int b_lo = min(tid * per_thread, seqs), b_hi = min(b_lo + per_thread, seqs);
  long long blocks = 0, units = 0;
  bool wrong = false;
  for (int b = b_lo; b < b_hi; ++b) {
    const TileSeq<SIDE> s(p, b, qu);
    const int c1 = s.q0 + s.n;
    const bool w = SIDE ? PartSeq(p, b).wrong(p, s.q0, s.n, s.len) : s.q0 < 0 || s.n < 0 || c1 < 0 || s.n > p.max_q || s.len < 0 || s.len > p.max_len ||
                   (p.causal && s.n > s.len) || (b == 0 && s.q0 != 0) || (b == p.B - 1 && c1 != p.total_q);
    wrong |= w;
    if (!w) {
      blocks += s.blocks_before(p, qu, s.units);
      units += s.units;
    }
  }
  long long blocks_to = blocks, units_to = units;      // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, blocks_to, o), w = __shfl_up_sync(0xffffffffu, units_to, o);
    if (lane >= o) {
      blocks_to += v;
      units_to += w;
    }
  }
  if (lane == 31) {
    sums[2 * warp] = blocks_to;
    sums[2 * warp + 1] = units_to;
  }
  const bool bad = __syncthreads_or(wrong) != 0;
  if (tid == 0) {
    *rec = make_int4(0, 0, 0, 0);            // no unit cut, unless found below
    if (bad) atomicExch(p.status, DEV_BAD_OFFSETS);
    if (SIDE && p.side != SIDE_IN && blockIdx.x == 0) *p.side_bad = bad;
  }
  if (bad || (SIDE && p.side == SIDE_IN && *p.side_bad)) return;
  blocks_to -= blocks;
  units_to -= units;
  long long all_blocks = 0, all_units = 0;
#pragma unroll
  for (int w = 0; w < kTThreads / 32; ++w) {
    if (w < warp) {
      blocks_to += sums[2 * w];
      units_to += sums[2 * w + 1];
    }
    all_blocks += sums[2 * w];
    all_units += sums[2 * w + 1];
  }
  // Few blocks per CTA: what counts is the longest run of blocks, not the sum of the work.
  const int cost = (int)min((long long)kUnitCost, all_blocks * p.Hkv / gridDim.x / 4);
  const long long total = (all_blocks + cost * all_units) * p.Hkv;
  const long long before = (blocks_to + cost * units_to) * p.Hkv, mine = (blocks + cost * units) * p.Hkv;
  const long long run = max((total + gridDim.x - 1) / gridDim.x, 2LL);
  const long long rs = run * blockIdx.x, re = min(rs + run, total);
  if (rs >= total) return;
  if (before <= rs && rs < before + mine) {
    int b = b_lo;
    long long at = before;
    for (;;) {
      const TileSeq<SIDE> s(p, b, qu);
      auto steps_before = [&](int rt) -> long long { return s.blocks_before(p, qu, rt) + (long long)rt * cost; };
      const long long per_head = steps_before(s.units);
      if (rs < at + per_head * p.Hkv) {
        const int h = (int)((rs - at) / per_head);
        at += h * per_head;
        int lo = 0, hi = s.units - 1;                  // the last rt whose first step is <= rs
        while (lo < hi) {
          const int mid = lo + (hi - lo + 1) / 2;
          if (at + steps_before(mid) <= rs) lo = mid;
          else hi = mid - 1;
        }
        misc[0] = b;
        misc[1] = h;
        misc[2] = lo;
        misc[3] = at + steps_before(lo);
        break;
      }
      at += per_head * p.Hkv;
      ++b;
    }
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int page_shift = 31 - __clz(p.page);
  auto table_of = [&](const UnitDesc& U) -> const int* {
    if constexpr (SIDE) {
      const PartSeq s(p, U.b);
      return s.table + (long long)s.b * s.max_pages;
    } else {
      return p.table + (long long)U.b * p.max_pages;
    }
  };
  // The roles' view of unit u: wait for its descriptor, and hand it back (one lane per warp).
  auto unit_ready = [&](uint32_t u) -> bool { return mbar_wait(BAR(T_UFULL + u % kUnitSlots), (u / kUnitSlots) & 1, wc); };
  // Release barrier of a product group, and its phase.
  auto rel = [&](uint32_t group) -> uint32_t { return BAR(T_REL + group % C::RELS); };
  auto rel_phase = [&](uint32_t group) -> uint32_t { return group / C::RELS & 1; };
  auto unit_done = [&](uint32_t u) { mbar_arrive(BAR(T_UFREE + u % kUnitSlots)); };

  // Register split against the launch's 128 x 512: producer, MMA, scheduler 64; softmax 184 each;
  // V and epilogue 80.
  if (wg == 0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0) {
      // ---------------------------------------------------------------- producer
      // Lane i < 128 / page loads the box of page i of a block (lane 0 alone when a page holds it).
      const int boxes = max(1, 128 >> page_shift), box_keys = min(p.page, 128);
      const uint32_t box_bytes = box_keys * D;
      uint32_t n_k = 0, n_v = 0;             // K, V blocks loaded so far
      uint32_t group = 0, g[C::NK] = {};     // product group of the next block's S; of the last blocks'
      bool ok = true;
      for (uint32_t nu = 0; ok; ++nu) {
        if (!__all_sync(0xffffffffu, unit_ready(nu))) { ok = false; break; }
        const UnitDesc& U = desc[nu % kUnitSlots];
        const int nmax = U.nmax, key0 = U.kt0 * 128 + lane * box_keys, len = U.len, h = U.h;
        const int* table = table_of(U);
        __syncwarp();
        if (lane == 0) unit_done(nu);
        if (nmax < 0) break;
        auto page_of = [&](int j) -> int {
          const int key = key0 + j * 128;
          if (lane >= boxes || j >= nmax || key >= len) return -1;
          const int pg = __ldg(table + (key >> page_shift));
          if (pg < 0 || pg >= p.num_pages) {
            atomicExch(p.status, DEV_BAD_PAGE);
            return 0;                        // any page of the cache: the sequence's results are undefined
          }
          return pg;
        };
        int pg_next = page_of(0);
        for (int j = 0; j < nmax; ++j) {
          const int pg = pg_next;
          pg_next = page_of(j + 1);
          const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, pg >= 0)) * box_bytes;
          const int z = pg * p.Hkv + h;
          const int ks = (int)(n_k % C::NK), vs = (int)(n_v % C::NV8);
          // The slot's block, NK before this one, was read by the products of group g[NK - 1].
          if (n_k >= C::NK && !warp_wait(rel(g[C::NK - 1]), rel_phase(g[C::NK - 1]), wc)) { ok = false; break; }
#pragma unroll
          for (int i = C::NK - 1; i > 0; --i) g[i] = g[i - 1];
          g[0] = group++;
          if (n_k > 0 || !p.test_skip_first_kv) {
            if (lane == 0) mbar_arrive_expect_tx(BAR(T_KFULL + ks), bytes);
            __syncwarp();
            if (pg >= 0) tma_load_3d(sbase + C::OFF_K + ks * C::K8 + lane * box_bytes, &tm_k, 0, 0, z, BAR(T_KFULL + ks));
          }
          ++n_k;
          if (n_v >= C::NV8 && !warp_wait(BAR(T_V8FREE + vs), (n_v / C::NV8 - 1) & 1, wc)) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(BAR(T_V8FULL + vs), bytes);
          __syncwarp();
          if (pg >= 0) tma_load_3d(sbase + C::OFF_V8 + vs * C::K8 + lane * box_bytes, &tm_v, 0, 0, z, BAR(T_V8FULL + vs));
          ++n_v;
        }
        if (nmax > 0) group += LAG;          // the last PVs are groups of their own
      }
      // Every copy has landed before the shared memory goes away, also when a wait ran out.
      if (lane == 0) {
        const unsigned long long t0 = globaltimer_ns();
        for (uint32_t i = n_k > C::NK ? n_k - C::NK : 0; i < n_k; ++i)
          while (!mbar_try_wait(BAR(T_KFULL + (i % C::NK)), (i / C::NK) & 1) && globaltimer_ns() - t0 < drain_ns(p)) {
          }
        for (uint32_t i = n_v > C::NV8 ? n_v - C::NV8 : 0; i < n_v; ++i)
          while (!mbar_try_wait(BAR(T_V8FULL + (i % C::NV8)), (i / C::NV8) & 1) && globaltimer_ns() - t0 < drain_ns(p)) {
          }
      }
    } else if (warp <= 2) {
      // ---------------------------------------------------------------- MMA issuers, one per tile
      // Group j of a unit: PV of block j - 1 (SPLIT: j - 2) and S of block j.
      if (lane == 0) {
        const int t = warp - 1;
        bool ok = true;
        uint32_t nk = 0, nv = 0, np = 0, no = 0, group = 0;   // blocks, V blocks, P phases used; units with a PV
        uint32_t n_turn = 0;                 // SPLIT: turns taken
        bool turn = false;                   // SPLIT, tile 0: the last group was tile 1's
        uint32_t nq = 0;                     // SPLIT: units with keys (tile 1 may have none of them)
        constexpr uint32_t HI = sdesc_sw128_hi(1024);
        const uint32_t tS = tmem + uint32_t(t * 128), tO = tmem + 256u + uint32_t(t * 128);
        const uint32_t q_lo = sdesc_sw128_lo(sbase + C::OFF_Q + (SPLIT ? 0 : 2 * t * C::Q8), 16);
        for (uint32_t nu = 0; ok; ++nu) {
          if (!unit_ready(nu)) { ok = false; break; }
          const UnitDesc& U = desc[nu % kUnitSlots];
          const int nmax = U.nmax, n_t = U.nt[t];
          unit_done(nu);
          if (nmax < 0) break;
          if (nmax == 0) continue;
          const uint32_t q_phase = SPLIT ? nq++ : no;
          for (int j = 0; j < nmax + LAG; ++j, ++group) {
            const bool pv = SPLIT ? j >= 2 && (j & 1) == t : j >= 1 && j <= n_t;
            const bool sp = SPLIT ? j < nmax && (j & 1) == t : j < n_t;
            const int j_own = SPLIT ? j >> 1 : j;      // step of this tile
            if (SPLIT && (j & 1) != t) {               // the other tile's group
              if (j >= LAG) ++nv;
              if (j < nmax) ++nk;
              continue;
            }
            const uint32_t vs = nv % C::NV16, ks = nk % C::NK;
            // P is the last to come.  (K also for a tile through with its blocks: it must not run ahead of the other.)
            if (j < nmax && !mbar_wait(BAR(T_KFULL + ks), (nk / C::NK) & 1, wc)) { ok = false; break; }
            if (j_own == 0 && sp && !mbar_wait(BAR(T_Q + (SPLIT ? 0 : t)), q_phase & 1, wc)) { ok = false; break; }
            if (pv) {
              if (j_own == 1 && no > 0 && !mbar_wait(BAR(T_OFREE + t), (no - 1) & 1, wc)) { ok = false; break; }
              if (!mbar_wait(BAR(T_V16FULL + vs), (nv / C::NV16) & 1, wc)) { ok = false; break; }
              if (!mbar_wait(BAR(T_PHALF + t), np & 1, wc)) { ok = false; break; }
            }
            // Tile 0's products of a group go before tile 1's: left alone, the tiles fall into step and
            // tensor cores and exponentials take turns instead of overlapping.
            // SPLIT: a group belongs to one tile; the unit's first is tile 0's, whoever had the last one.
            if constexpr (SPLIT) {
              if (j > 0 || turn) {
                if (!mbar_wait(BAR(T_TURN + t), n_turn & 1, wc)) { ok = false; break; }
                ++n_turn;
              }
            } else {
              if (!mbar_wait(BAR(T_TURN + t), (group + 1 - t) & 1, wc)) { ok = false; break; }
            }
            tc_fence_after();
            if (pv) {
              // O_t += P_t V16, A = P from tensor memory (f16 pairs)
              const uint32_t v_lo = sdesc_sw128_lo(sbase + C::OFF_V16 + vs * C::V16, C::CH16);
              // The first half of the keys while the softmax works on the second.
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_ts_w(tO, tS + kk * 8, v_lo + kk * (2048 >> 4), HI, C::IDESC_PV, (j_own > 1 || kk > 0) ? 1u : 0u);
              if (!mbar_wait(BAR(T_PFULL + t), np & 1, wc)) { ok = false; break; }
              ++np;
              tc_fence_after();
#pragma unroll
              for (int kk = 4; kk < 8; ++kk) mma_ts_w(tO, tS + kk * 8, v_lo + kk * (2048 >> 4), HI, C::IDESC_PV, 1u);
              if (j_own == n_t) {
                mma_commit(BAR(T_OFULL + t));
                ++no;
              }
            }
            if (sp) {
              // S_t = (Q1_t + Q2_t) K8_j^T, K = 32 columns a step
              const uint32_t k_lo = sdesc_sw128_lo(sbase + C::OFF_K + ks * C::K8, 16);
#pragma unroll
              for (int kk = 0; kk < 2 * (D / 32); ++kk)
                mma_ss_f8_w(tS, q_lo + (((kk / (D / 32)) * C::Q8 + (kk % (D / 32)) * 32) >> 4), C::QK_HI,
                            k_lo + ((kk % (D / 32)) * 32 >> 4), C::QK_HI, kk < D / 32 ? C::IDESC_Q1K : C::IDESC_Q2K,
                            kk > 0 ? 1u : 0u);
            }
            if (SPLIT) turn = j + 1 < nmax + LAG || t > 0;
            if (!SPLIT || turn) mbar_arrive(BAR(T_TURN + 1 - t));
            if (sp) mma_commit(BAR(T_SFULL + t));
            mma_commit(rel(group));
            if (j >= LAG) ++nv;
            if (j < nmax) ++nk;
          }
        }
        mma_commit(BAR(T_DONE + t));
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(BAR(T_DONE + t), 0) && globaltimer_ns() - t0 < drain_ns(p)) {
        }
      }
    } else if (warp == 3) {
      // ---------------------------------------------------------------- scheduler
      // Walks the CTA's units; steps are counted from the CTA's first.
      if (lane == 0) {
        int b = (int)misc[0], h = (int)misc[1], rt = (int)misc[2], ubeg = (int)(misc[3] - rs);
        const int end = (int)(re - rs), step_run = (int)run;
        TileSeq<SIDE> sq(p, b, qu);
        bool first = true;
        for (uint32_t nu = 0;;) {
          const int uend = ubeg + cost + sq.blocks(p, qu, rt);
          // The unit's blocks here; none where the run ends in a unit's first steps, or starts behind its last.
          const int kt0 = max(0, -ubeg - cost), kt1 = min(uend, end) - ubeg - cost;
          const bool over = ubeg >= end;
          if (over || kt1 > kt0) {
            if (nu >= kUnitSlots && !mbar_wait(BAR(T_UFREE + nu % kUnitSlots), (nu / kUnitSlots - 1) & 1, wc)) break;
            UnitDesc& U = desc[nu % kUnitSlots];
            if (over) {
              U.nmax = -1;
              mbar_arrive(BAR(T_UFULL + nu % kUnitSlots));
              break;
            }
            const int rows = min(qu, sq.n - rt * qu) * p.g;
            int nt[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int r = min(rows, (t + 1) * 128) - t * 128;           // rows of the tile
              const int lim = r > 0 ? (sq.causal ? sq.len - sq.n + rt * qu + (t * 128 + r - 1) / p.g + 1 : sq.len) : 0;
              nt[t] = max(0, min((lim + 127) / 128, kt1) - kt0);
            }
            U.nmax = max(nt[0], nt[1]);
            U.nt[0] = SPLIT ? (nt[0] + 1) / 2 : nt[0];
            U.nt[1] = SPLIT ? nt[0] / 2 : nt[1];
            U.kt0 = kt0;
            U.len = sq.len;
            U.b = b;
            U.h = h;
            U.rows = rows;
            U.q0 = sq.q0 + rt * qu;
            U.lim0 = sq.causal ? sq.len - sq.n + rt * qu + 1 : sq.len;
            if constexpr (SIDE) {
              U.causal = sq.causal;
              U.part = b >= p.B ? 1 : 0;
            }
            U.whole = kt0 == 0 && uend <= end ? 1 : 0;
            U.second = first ? 0 : 1;
            U.more = kt0 == 0 ? (uend - 1) / step_run : -1;   // cut: the CTAs behind this one that go on with it
            first = false;
            mbar_arrive(BAR(T_UFULL + nu % kUnitSlots));
            ++nu;
          }
          ubeg = uend;
          if (ubeg >= end) continue;
          if (++rt >= sq.units) {
            rt = 0;
            if (++h == p.Hkv) {
              h = 0;
              do sq = TileSeq<SIDE>(p, ++b, qu);   // steps are left: there is another unit
              while (sq.units == 0);
            }
          }
        }
      }
    }
  } else if (wg == 1 || wg == 2) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    // ------------------------------------------------------------------ softmax
    const int t = wg - 1;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t tS = tmem + (uint32_t((warp & 3) * 32) << 16) + uint32_t(t * 128);
    const int row0 = SPLIT ? 0 : t * 128, r = row0 + row, qi = r / p.g;      // row of the unit, its query
    constexpr int STRIDE = SPLIT ? 256 : 128;          // keys from one of a tile's blocks to the next
    uint32_t ns = 0, ns_other = 0;           // S phases used; SPLIT: by tile 1
    bool ok = true;
    for (uint32_t nu = 0; ok; ++nu) {
      if (!__all_sync(0xffffffffu, unit_ready(nu))) { ok = false; break; }
      const UnitDesc& U = desc[nu % kUnitSlots];
      const int n_t = U.nt[t], kt0 = U.kt0 + (SPLIT ? t : 0), len = U.len, h = U.h, q0 = U.q0;
      const int n_other = SPLIT ? U.nt[1] : 0;
      const bool more = U.nmax >= 0, live = r < U.rows;
      const int* table = table_of(U);
      const bool causal = SIDE ? U.causal != 0 : p.causal != 0;
      const int lim = (causal && live ? U.lim0 + qi : len) - kt0 * 128;                       // visible keys of this row,
      const int min_lim = (causal ? U.lim0 + row0 / p.g : len) - kt0 * 128;                // of the tile's first row
      __syncwarp();
      if (lane == 0) unit_done(nu);
      if (!more) break;
      float c_row = 0.f;
      if (n_t > 0) {
        // Q is free: every S of the unit before has been waited for (SPLIT: tile 1's too).  Each warp brings its
        // 32 rows, whole rows at a time (D / 8 lanes of 16 bytes each), QB steps' loads under way at once.
        constexpr int LPR = D / 8, RPS = 32 / LPR, QB = 4;          // lanes per row, rows per step
        // (rows that are not in use take the unit's first: loads without conditions).
        const long long at = live ? ((long long)(r - qi * p.g) * p.total_q + qi) * D : 0;    // this lane's own row
        const uint16_t* base = static_cast<const uint16_t*>(p.q) + ((long long)h * p.g * p.total_q + q0) * D + lane % LPR * 8;
        uint8_t* q1 = smem + C::OFF_Q + (SPLIT ? 0 : 2 * t * C::Q8) + (warp & 3) * 32 * D;
        if constexpr (SPLIT) {
          if (t == 0 && ns_other > 0 && !warp_wait(BAR(T_SFULL + 1), (ns_other - 1) & 1, wc)) { ok = false; break; }
        }
        uint32_t e_own = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < 32 / RPS; i0 += QB) {
          uint4 w[QB];
#pragma unroll
          for (int k = 0; k < QB; ++k) {
            w[k] = __ldg(reinterpret_cast<const uint4*>(base + __shfl_sync(0xffffffffu, at, (i0 + k) * RPS + lane / LPR)));
          }
#pragma unroll
          for (int k = 0; k < QB; ++k) {
            const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
            float amax = 0.f;
#pragma unroll
            for (int x = 0; x < 4; ++x)
              amax = fmax3(amax, fabsf(__uint_as_float(u[x] << 16)), fabsf(__uint_as_float(u[x] & 0xffff0000u)));
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const uint32_t e = __float_as_uint(amax) >> 23;        // biased exponent
            const uint32_t e_row = __shfl_sync(0xffffffffu, e, lane % RPS * LPR);
            if (lane / RPS == i0 + k) e_own = e_row;
            const bool usable = e >= 8 && e < 255;                 // else 0 or tiny: left as it is; infinite: NaN
            const float inv = usable ? __uint_as_float((254u + 7u - e) << 23) : 1.f;
            const uint32_t poison = e == 255 ? 0x7f7f7f7fu : 0u;
            uint32_t c1[2], c2[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float x0 = __uint_as_float(u[2 * x] << 16) * inv, x1 = __uint_as_float(u[2 * x] & 0xffff0000u) * inv;
              const float x2 = __uint_as_float(u[2 * x + 1] << 16) * inv, x3 = __uint_as_float(u[2 * x + 1] & 0xffff0000u) * inv;
              const uint32_t hq = to_e4m3x2(x0, x1) | (to_e4m3x2(x2, x3) << 16);
              float y0, y1, y2, y3;
              e4m3x4_to_f32(hq, y0, y1, y2, y3);
              c1[x] = hq | poison;
              c2[x] = to_e5m2x2(x0 - y0, x1 - y1) | (to_e5m2x2(x2 - y2, x3 - y3) << 16);
            }
            const int rw = (i0 + k) * RPS + lane / LPR, ch = lane % LPR;   // row of the warp's 32, 8-byte piece
            const int off = rw * D + (((ch >> 1) ^ (D == 128 ? (rw & 7) : ((rw >> 1) & 3))) << 4) + (ch & 1) * 8;
            if (SPLIT && t > 0) continue;    // tile 1 wants the rows' factors only
            *reinterpret_cast<uint2*>(q1 + off) = make_uint2(c1[0], c1[1]);
            *reinterpret_cast<uint2*>(q1 + C::Q8 + off) = make_uint2(c2[0], c2[1]);
          }
        }
        c_row = p.c * (e_own >= 8 && e_own < 255 ? __uint_as_float((e_own - 7u) << 23) : 1.f);
        fence_proxy_async_smem();            // generic writes -> tensor-core reads
        if (!SPLIT || t == 0) mbar_arrive(BAR(T_Q + t));
      }
      if constexpr (SPLIT) ns_other += n_other;
      // K scales: lane % NG looks after a group of KG keys (all lanes after the one page when NG = 1);
      // pages one block further ahead than scales.
      auto page_of = [&](int j) -> int {
        const int key = kt0 * 128 + j * STRIDE + (NG > 1 ? lane % NG * KG : 0);
        if (j >= n_t || key >= len) return -1;
        const int pg = __ldg(table + (key >> page_shift));
        return (unsigned)pg < (unsigned)p.num_pages ? pg : 0;
      };
      auto scale_of = [&](int pg) -> float { return pg >= 0 ? __ldg(p.k_scale + (long long)pg * p.Hkv + h) : 0.f; };
      float sk_next = scale_of(page_of(0));
      int pg_next = page_of(1);
      // The V scales too: when the largest so far grows, O is rescaled like for a maximum.
      auto v_scale_of = [&](int pg) -> float { return pg >= 0 ? __ldg(p.v_scale + (long long)pg * p.Hkv + h) : 0.f; };
      float sv_next = v_scale_of(page_of(0));
      float m = -INFINITY, l = 0.f, rref = kMinScale;
      for (int j = 0; j < n_t; ++j) {
        const float sk = sk_next;
        float vmax = sv_next;
        sk_next = scale_of(pg_next);
        sv_next = v_scale_of(pg_next);
        pg_next = page_of(j + 2);
        if constexpr (NG > 1) {
#pragma unroll
          for (int o = NG / 2; o > 0; o >>= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, o));
        }
        float fac[NG];
#pragma unroll
        for (int i = 0; i < NG; ++i)
          fac[i] = fmaxf(c_row * (NG > 1 ? __shfl_sync(0xffffffffu, sk, i) : sk), kMinFactor);
        if (!warp_wait(BAR(T_SFULL + t), ns & 1, wc)) { ok = false; break; }
        ++ns;
        tc_fence_after();
        uint32_t u[128];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(tS + q * 32, *reinterpret_cast<uint32_t(*)[32]>(&u[q * 32]));
        tmem_wait_ld();
        reg_fence(u);
        float* s = reinterpret_cast<float*>(u);
        if (j * STRIDE + 128 > min_lim) {
          const int vis = lim - j * STRIDE;     // visible columns
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i >= vis) s[i] = -INFINITY;
        }
        float rmax = -INFINITY;
        if constexpr (NG == 1) {
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int i = 4; i < 124; i += 8) {
            mx[0] = fmax3(mx[0], s[i], s[i + 1]);
            mx[1] = fmax3(mx[1], s[i + 2], s[i + 3]);
            mx[2] = fmax3(mx[2], s[i + 4], s[i + 5]);
            mx[3] = fmax3(mx[3], s[i + 6], s[i + 7]);
          }
          mx[0] = fmax3(mx[0], s[124], s[125]);
          mx[1] = fmax3(mx[1], s[126], s[127]);
          rmax = fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * fac[0];
        } else {
#pragma unroll
          for (int gq = 0; gq < NG; ++gq) {
            const float* x = s + gq * KG;
            float a = fmax3(x[0], x[1], x[2]), b = fmax3(x[3], x[4], x[5]);
#pragma unroll
            for (int i = 6; i < KG - 2; i += 4) {
              a = fmax3(a, x[i], x[i + 1]);
              b = fmax3(b, x[i + 2], x[i + 3]);
            }
            rmax = fmaxf(rmax, fmax3(fmaxf(a, b), x[KG - 2], x[KG - 1]) * fac[gq]);
          }
        }
        const float m_cand = fmaxf(m, rmax);
        float alpha = 1.f;
        if (j == 0) {
          m = m_cand;
        } else if (m_cand - m > kTau) {
          alpha = ex2_mufu(m - m_cand);
          m = m_cand;
        }
        // Rare after the first blocks.  S_t(j) complete: PV_t(j - 1), issued before it, is too.
        const float scale_o = vmax > rref ? alpha * (rref / vmax) : alpha;
        rref = fmaxf(rref, vmax);
        if (j > 0 && __any_sync(0xffffffffu, scale_o != 1.f)) {
#pragma unroll 1
          for (int q = 0; q < D / 16; ++q) {
            uint32_t x[16];
            tmem_ld16(tS + 256u + q * 16, x);   // O_t lies 256 columns behind S_t
            tmem_wait_ld();
            reg_fence(x);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * scale_o);
            tmem_st16(tS + 256u + q * 16, x);
          }
        }
        const float off = kPShift - (m == -INFINITY ? 0.f : m);
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 64 * hf; i < 64 * hf + 64; i += 2) {
            float x0, x1;
            ffma2_bc(x0, x1, s[i], s[i + 1], fac[i / KG], off);
            const float e0 = ex2_mufu(x0), e1 = ex2_mufu(x1);
            pk[(i >> 1) & 31] = pack_f16x2(e0, e1);
            const int a2 = ((i >> 1) & 1) * 2;
            fadd2(acc[a2], acc[a2 + 1], acc[a2], acc[a2 + 1], e0, e1);
          }
          tmem_st32(tS + hf * 32, pk);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(BAR((hf ? T_PFULL : T_PHALF) + t));
        }
        l = l * alpha + ((acc[0] + acc[1]) + (acc[2] + acc[3]));
      }
      // The statistics of the unit before have been read.  (This also keeps a tile without rows
      // from running ahead of the other roles.)
      if (ok && nu > 0 && !warp_wait(BAR(T_EPI), (nu - 1) & 1, wc)) ok = false;
      if (!ok) break;
      float* out = fin + t * 384 + row;
      out[0] = m;
      out[128] = l;
      out[256] = rref;
      mbar_arrive(BAR(T_FIN + t));
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    // ------------------------------------------------------------------ V, epilogue
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const int ct = tid - 384, w4 = ct >> 5;
    uint32_t group = 0, g1 = 0, g2 = 0;      // product group of the next block's S; of the last two blocks' PV
    uint32_t nv = 0, nof0 = 0, nof1 = 0;     // V blocks widened; per tile O phases used
    bool ok = true;
    for (uint32_t nu = 0; ok; ++nu) {
      if (!__all_sync(0xffffffffu, unit_ready(nu))) { ok = false; break; }
      const UnitDesc& U = desc[nu % kUnitSlots];
      const int nmax = U.nmax, nt0 = U.nt[0], nt1 = U.nt[1], kt0 = U.kt0, len = U.len, h = U.h;
      const int* table = table_of(U);
      const int part_of_keys = SIDE ? U.part : 0;
      if (nmax < 0) break;                   // the last descriptor is not reused
      float rref = kMinScale;                // largest V scale so far
      float rref_other = kMinScale;          // SPLIT: of the other tile's blocks (they take turns)
      auto page_of = [&](int j) -> int {
        const int key = (kt0 + j) * 128 + (NG > 1 ? lane % NG * KG : 0);
        if (j >= nmax || key >= len) return -1;
        const int pg = __ldg(table + (key >> page_shift));
        return (unsigned)pg < (unsigned)p.num_pages ? pg : 0;
      };
      auto scale_of = [&](int pg) -> float { return pg >= 0 ? __ldg(p.v_scale + (long long)pg * p.Hkv + h) : 0.f; };
      float sv_next = scale_of(page_of(0));
      int pg_next = page_of(1);
      // Results of the unit before were staged in the V16 slots, each warp's on its own: all have left.
      if (nu > 0 && !warp_wait(BAR(T_EPI), (nu - 1) & 1, wc)) { ok = false; break; }
      // The first block here with keys that some of the unit's queries do not see.
      const int j_hid = U.lim0 < len ? (U.lim0 >> 7) - kt0 : nmax;
      if (ct < D) nan_keys[(~nu & 1) * D + ct] = kNoKey;           // the next unit's (the one before has been read)
      if (ct == 0) any_nan[~nu & 1] = 0;
      // V8 block -> f16 in the layout the PV product reads (64-column boxes, 128-byte swizzle).  Thread
      // pieces of 16 codes; each quarter-warp takes half of two adjacent 128-byte lines, so that its
      // loads and each of its two rounds of stores fall on eight distinct bank groups.
      auto widen = [&](int j, auto check) -> bool {
        const float sv = sv_next;
        sv_next = scale_of(pg_next);
        pg_next = page_of(j + 2);
        float vmax = sv;
        if constexpr (NG > 1) {
#pragma unroll
          for (int o = NG / 2; o > 0; o >>= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, o));
        }
        if constexpr (SPLIT) {
          const float x = rref;
          rref = rref_other;
          rref_other = x;
        }
        rref = fmaxf(rref, vmax);
        const float wgt = sv / rref * kVShift;
        const uint32_t w_mine = pack_f16x2(wgt, wgt);  // this lane's group's factor
        const uint32_t vs8 = nv % C::NV8, vs16 = nv % C::NV16;
        if (!warp_wait(BAR(T_V8FULL + vs8), (nv / C::NV8) & 1, wc)) return false;
        // The slot's block, two before this one, was read by the products of group g2.
        if (nv >= C::NV16 && !warp_wait(rel(g2), rel_phase(g2), wc)) return false;
        g2 = g1;
        g1 = group + LAG;                    // PV of block j
        ++group;
        const uint8_t* src = smem + C::OFF_V8 + vs8 * C::K8;
        uint8_t* dst = smem + C::OFF_V16 + vs16 * C::V16;
        const int left = len - (kt0 + j) * 128;                    // keys that exist
        const int quarter = lane >> 3, half = (lane & 7) >> 2;
        const int u = (lane & 3) + 4 * (half ^ (quarter & 1));     // 16-byte piece of a line
        const int r0 = 4 * w4 + 2 * (quarter >> 1) + half, sw = r0 & 7;   // line 16 it + r0
        const uint8_t* s_base = src + r0 * 128 + ((u ^ sw) << 4);
        // d = 128: a line is a key; d = 64: two keys.
        const auto key_of = [&](int it) { return D == 128 ? it * 16 + r0 : 2 * (it * 16 + r0) + (u >> 2); };
        if constexpr (decltype(check)::value) {
#pragma unroll 1
          for (int it = 0; it < D / 16; ++it) {
            const int key = len - left + key_of(it);
            uint8_t* piece = const_cast<uint8_t*>(s_base) + it * 2048;
            if (key < len && key >= U.lim0 && any_nan_code(*reinterpret_cast<const uint4*>(piece)))
              take_nan_codes(piece, key, nan_keys + (nu & 1) * D + (D == 128 ? u : u & 3) * 16, any_nan + (nu & 1));
          }
        }
#pragma unroll 4
        for (int it = 0; it < D / 16; ++it) {
          uint4 v = *reinterpret_cast<const uint4*>(s_base + it * 2048);
          const int key = key_of(it);
          uint32_t wv = w_mine;
          if constexpr (NG > 1) wv = __shfl_sync(0xffffffffu, w_mine, (D == 128 ? it : 2 * it + (w4 >> 1)) * 16 / KG);
          if (key >= left) v = make_uint4(0u, 0u, 0u, 0u);         // whatever the codes are (NaN too)
          const uint32_t in[4] = {v.x, v.y, v.z, v.w};
          uint32_t hh[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            hh[2 * i] = hmul2(e4m3x2_f16x2(in[i]), wv);
            hh[2 * i + 1] = hmul2(e4m3x2_f16x2_hi(in[i]), wv);
          }
          const int q = u & 3;                                     // pieces 2q, 2q + 1 of the f16 row
          uint8_t* d_row = dst + (D == 128 ? (u >> 2) * C::CH16 : 0u) + key * 128;
          const int ks = key & 7;
          *reinterpret_cast<uint4*>(d_row + (((2 * q) ^ ks) << 4)) = make_uint4(hh[0], hh[1], hh[2], hh[3]);
          *reinterpret_cast<uint4*>(d_row + (((2 * q + 1) ^ ks) << 4)) = make_uint4(hh[4], hh[5], hh[6], hh[7]);
        }
        fence_proxy_async_smem();            // generic writes -> tensor-core reads
        mbar_arrive(BAR(T_V16FULL + vs16));
        mbar_arrive(BAR(T_V8FREE + vs8));
        ++nv;
        return true;
      };
      // Two loops, so that the blocks that all queries see carry nothing of the check for NaN codes (with
      // one loop prompts of 4096 took 3.5 % longer).
      int j = 0;
      for (const int j_end = min(j_hid, nmax); ok && j < j_end; ++j) ok = widen(j, std::false_type());
      for (; ok && j < nmax; ++j) ok = widen(j, std::true_type());
      if (!ok) break;
      if (nmax > 0) group += LAG;            // the groups of the unit's last PVs
      // Epilogue per tile: O / l to its rows, or O and the statistics to the workspace.
      const bool whole = U.whole != 0;
      const int part = 2 * blockIdx.x + U.second, rows = U.rows, q0 = U.q0;
      if (U.more > 0 && !whole && ct == 0) *rec = make_int4(h | part_of_keys << 30, q0, rows / p.g, 2 * U.more + U.second);
      // Every product of both tiles is complete: O is final and V16 is free.
      if (nt0 > 0 && !warp_wait(BAR(T_OFULL), nof0++ & 1, wc)) { ok = false; break; }
      if (nt1 > 0 && !warp_wait(BAR(T_OFULL + 1), nof1++ & 1, wc)) { ok = false; break; }
      if constexpr (SPLIT) {                 // tile 1's share of the keys into tile 0
        if (!warp_wait(BAR(T_FIN), nu & 1, wc) || !warp_wait(BAR(T_FIN + 1), nu & 1, wc)) { ok = false; break; }
        if (nt1 > 0) {
          tc_fence_after();
          float* st = fin + row;
          const float m = fmaxf(st[0], st[384]), mu = m == -INFINITY ? 0.f : m, ref = fmaxf(st[256], st[640]);
          const float w0 = ex2_mufu(st[0] - mu), w1 = ex2_mufu(st[384] - mu);
          const float f0 = w0 * (st[256] / ref), f1 = w1 * (st[640] / ref);
          st[128] = st[128] * w0 + st[512] * w1;
          st[0] = m;
          st[256] = ref;
          const uint32_t tO = tmem + lane_off + 256u;
#pragma unroll 1
          for (int q = 0; q < D / 16; ++q) {
            uint32_t x[16], y[16];
            tmem_ld16(tO + q * 16, x);
            tmem_ld16(tO + 128u + q * 16, y);
            tmem_wait_ld();
            reg_fence(x);
            reg_fence(y);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f0 + __uint_as_float(y[i]) * f1);
            tmem_st16(tO + q * 16, x);
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(BAR(T_OFREE + 1));
        }
      }
#pragma unroll 1
      for (int t = 0; t < (SPLIT ? 1 : 2); ++t) {
        const int n_t = t ? nt1 : nt0;
        if (!SPLIT && !warp_wait(BAR(T_FIN + t), nu & 1, wc)) { ok = false; break; }
        tc_fence_after();
        const float* st = fin + t * 384 + row;
        const float m = st[0], l = st[128], ref = st[256] / kVShift;
        const int r = t * 128 + row, qi = r / p.g;
        const bool live = r < rows;
        const long long orow = (long long)(h * p.g + (r - qi * p.g)) * p.total_q + q0 + qi;
        const long long prow = (long long)part * kTRows + r;
        float inv = whole ? (l == 0.f ? 0.f : ref / l) : 1.f, lse2 = m - kPShift + __log2f(l), w_side = 0.f;
        const long long pieces = (long long)p.total_q * p.g;       // from one piece of 4 columns to the next
        float4* side = side_piece<D>(p, part_of_keys, h, q0, r, 0);              // (used where the row is live)
        if (whole && live && SIDE && p.side == SIDE_IN) {
          const float2 w = join_side(p, side_row(p, h, q0, r), lse2, lse2);
          inv *= w.x;
          w_side = w.y;
        }
        const uint32_t tO = tmem + lane_off + 256u + uint32_t(t * 128);
        // Whole units go through shared memory (V16 slot t: no product reads it any more), so that rows
        // leave in whole lines; a warp stages its own 32 rows.
        uint8_t* stage = smem + C::OFF_V16 + t * C::V16 + (warp & 3) * 32 * (2 * D);
        bool done = false;
        if constexpr (SIDE) {
          if (whole) {                       // 16 columns at a time: more would spill
            done = true;
            float4* at = side;
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              uint32_t x[16];
              float4 z[4];
              if (p.side == SIDE_IN) {
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = live ? at[i * pieces] : make_float4(0.f, 0.f, 0.f, 0.f);
              }
              if (n_t > 0) {
                tmem_ld16(tO + q * 16, x);
                tmem_wait_ld();
                reg_fence(x);
              } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = 0u;
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float4 y = make_float4(__uint_as_float(x[4 * i]) * inv, __uint_as_float(x[4 * i + 1]) * inv,
                                       __uint_as_float(x[4 * i + 2]) * inv, __uint_as_float(x[4 * i + 3]) * inv);
                if (p.side != SIDE_IN) {
                  if (live) at[i * pieces] = y;
                  continue;
                }
                y = make_float4(y.x + w_side * z[i].x, y.y + w_side * z[i].y, y.z + w_side * z[i].z, y.w + w_side * z[i].w);
                *reinterpret_cast<uint2*>(stage + lane * (2 * D) + (((q * 2 + (i >> 1)) ^ (lane & 7)) << 4) + (i & 1) * 8) =
                    make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
              }
              at += 4 * pieces;
              __syncwarp();
            }
          }
        }
        uint32_t x[32];
#pragma unroll 1
        for (int q = 0; q < D / 32 && !done; ++q) {
          if (n_t > 0) {
            tmem_ld32(tO + q * 32, x);
            tmem_wait_ld();
            reg_fence(x);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = 0u;
          }
          if (!SIDE && whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t y[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                y[k] = pack_bf16x2(__uint_as_float(x[8 * i + 2 * k]) * inv, __uint_as_float(x[8 * i + 2 * k + 1]) * inv);
              *reinterpret_cast<uint4*>(stage + lane * (2 * D) + (((q * 4 + i) ^ (lane & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
            }
          } else if (live) {
            uint4* out = reinterpret_cast<uint4*>(ws + W.part) + ((long long)part * (D / 4) + q * 8) * kTRows + r;
#pragma unroll
            for (int i = 0; i < 8; ++i) out[i * kTRows] = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          }
          __syncwarp();
        }
        if (whole && !(SIDE && p.side != SIDE_IN)) {
          constexpr int LPR = D / 8, RPS = 32 / LPR;
          const long long mine = live ? orow : -1;
#pragma unroll 4
          for (int i = 0; i < 32 / RPS; ++i) {
            const int rw = i * RPS + lane / LPR;
            const long long a = __shfl_sync(0xffffffffu, mine, rw);
            const uint4 v = *reinterpret_cast<const uint4*>(stage + rw * (2 * D) + (((lane % LPR) ^ (rw & 7)) << 4));
            if (a >= 0) *(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + a * D) + lane % LPR) = v;
          }
          __syncwarp();
        }
        if (n_t > 0) {
          tc_fence_before();
          mbar_arrive(BAR(T_OFREE + t));
        }
        if (any_nan[nu & 1] && live) {       // (then the unit is causal; the lanes' stores above came before)
#pragma unroll 1
          for (int i = 0; i < D; ++i) {
            if (nan_keys[(nu & 1) * D + i] >= U.lim0 + qi) continue;
            if (whole && SIDE && p.side != SIDE_IN) reinterpret_cast<float*>(side + (i / 4) * pieces)[i % 4] = __int_as_float(0x7fffffff);
            else if (whole) static_cast<uint16_t*>(p.o)[orow * D + i] = 0x7fff;
            else reinterpret_cast<uint32_t*>(ws + W.part)[(((long long)part * (D / 4) + i / 4) * kTRows + r) * 4 + i % 4] = 0x7fffffffu;
          }
        }
        if (live) {
          if (whole && SIDE && p.side != SIDE_IN) p.side_lse[part_of_keys][side_row(p, h, q0, r)] = lse2;
          else if (whole) p.lse[orow] = lse2 * kLn2;
          else reinterpret_cast<float4*>(ws + W.stat)[prow] = make_float4(m - kPShift, l, ref, 0.f);
        }
      }
      if (!ok) break;
      mbar_arrive(BAR(T_EPI));
      __syncwarp();
      if (lane == 0) unit_done(nu);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int NG, bool SPLIT, bool SIDE>
cudaError_t launch_tile(const CacheMaps& maps, const CacheParams& p, int grid, cudaStream_t s) {
  using C = TileCfg<D, SPLIT>;
  static std::once_flag flags[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::call_once(flags[dev & 63], [&] {
    attr_err[dev & 63] = cudaFuncSetAttribute(fwd_cache_tile_kernel<D, NG, SPLIT, SIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (attr_err[dev & 63] != cudaSuccess) return attr_err[dev & 63];
  // A dependent launch of whatever runs before: the kernel waits for it to be done, but is in place by then.
  e = launch_pdl(fwd_cache_tile_kernel<D, NG, SPLIT, SIDE>, dim3(grid), dim3(kTThreads), C::SMEM, s, maps.k, maps.v, p);
  if (e != cudaSuccess) return e;
  return launch_fwd_cache_merge(p, D, kTRows, grid, s);
}

}  // namespace

#if CACHE_TILE_SIDE
cudaError_t launch_fwd_cache_tile_side(const CacheMaps& maps, const CacheParams& p, int d, int sms, cudaStream_t s) {
#else
size_t cache_tile_workspace_bytes(int d, int sms) { return cache_ws(sms, kTRows, d).total; }

cudaError_t launch_fwd_cache_tile(const CacheMaps& maps, const CacheParams& p, int d, int sms, cudaStream_t s) {
  if (p.side != SIDE_NONE) return launch_fwd_cache_tile_side(maps, p, d, sms, s);
#endif
  // 16 sequences of 16000 keys, 128 rows per K/V head: 145 us against 203; 32 rows 141 against 198.
  const int max_q = p.side == SIDE_BOTH && p.two.max_q > p.max_q ? p.two.max_q : p.max_q;
  const bool split = (long long)max_q * p.g <= 128;
  auto go = [&](auto dim, auto groups) {
    constexpr bool side = CACHE_TILE_SIDE;
    return split ? launch_tile<dim, groups, true, side>(maps, p, sms, s) : launch_tile<dim, groups, false, side>(maps, p, sms, s);
  };
  using I1 = std::integral_constant<int, 1>;
  using I8 = std::integral_constant<int, 8>;
  using I64 = std::integral_constant<int, 64>;
  using I128 = std::integral_constant<int, 128>;
  using I2 = std::integral_constant<int, 2>;
  using I4 = std::integral_constant<int, 4>;
  // Two prompts of 4096 over pages of 128 / 64 / 32 / 16: 670 / 677 / 702 / 746 us (the middle two with eight groups: 741, 743).
  if (p.page == 128) return d == 64 ? go(I64(), I1()) : go(I128(), I1());
  if (p.page == 64) return d == 64 ? go(I64(), I2()) : go(I128(), I2());
  if (p.page == 32) return d == 64 ? go(I64(), I4()) : go(I128(), I4());
  return d == 64 ? go(I64(), I8()) : go(I128(), I8());
}

}  // namespace attn
