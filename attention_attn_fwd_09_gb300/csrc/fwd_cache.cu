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
// Lists (a unit is a query and its pages): 128 pages of 32 keys for each of 64 sequences 113 us in a graph,
// 4.7 TB/s; 64 pages for one 13 us, of the kernel's 12300 cycles 3300 the start, 2700 look-ups, 2300 the join.
// Behind shared prefixes: a unit's result is joined with the other part's, in the epilogue or by
// fwd_cache_join_kernel; 64 sequences' keys behind 32768 92 us in all, by tiles and then here.
//
// Numbers: q is scaled by a power of two per row (largest |q| in [2^14, 2^15)) and held in f16: exact
// down to 2^-31 of the row's largest component, off by at most 2^-39 of it below.  exp2(s - m + 14)
// <= 2^14 times the page's V scale over the largest V scale so far is rounded to f16 (11 bits, against
// 8 of a bf16 weight; the 2^14 keeps weights down to 2^-28 of the largest normal).  Scores, maxima,
// sums and O are fp32.
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "cache.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kPiece = 32;                   // keys per piece
constexpr int kSMs = 152;                  // blocks of the merge kernel are a multiple of these
constexpr float kShift = 14.f;               // weights are held times 2^14
// What starting and ending a unit counts for when work is cut, in pieces (a shared prefix before 64 sequences of up
// to 1024 keys: 90 us, without it 114; 6 and 20 alike).  attn_fwd_kv_fp8 counts pieces alone.
constexpr int kUnitCost = 12;

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

// What the kernel works on: sequences; queries with lists of pages (p.list); sequences whose keys come in two parts
// (p.side).  The latter two count what starting and ending a unit costs when they cut the work.
// KIND_LIST: a unit is one query and K/V head, its list's pages end to end in pieces.
enum : int { KIND_PLAIN = 0, KIND_LIST = 1, KIND_SIDE = 2 };

template <int KIND>
__device__ __forceinline__ int pieces_of(const CacheParams& p, int b) {
  int n, len;
  if constexpr (KIND == KIND_SIDE) {
    const PartSeq s(p, b);
    n = __ldg(s.cu + s.b + 1) - __ldg(s.cu + s.b);
    len = __ldg(s.lens + s.b);
  } else {
    n = __ldg(p.cu_q + b + 1) - __ldg(p.cu_q + b);
    len = __ldg(p.kv_lens + b);
  }
  return n > 0 ? max(1, (len + kPiece - 1) / kPiece) : 0;
}

// The sequence of packed query t: the last one that starts at or before it (decoding: its own number).
__device__ __forceinline__ int seq_of(const CacheParams& p, int t) {
  if (p.B == p.total_q && __ldg(p.cu_q + t) == t && __ldg(p.cu_q + t + 1) == t + 1) return t;
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (__ldg(p.cu_q + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
// Keys that query t of sequence b sees.
__device__ __forceinline__ int keys_seen(const CacheParams& p, int b, int t) {
  const int len = __ldg(p.kv_lens + b);
  return p.causal ? len - (__ldg(p.cu_q + b + 1) - 1 - t) : len;
}
// Pages it sees; as many entries of its list are read at most (they are distinct).
__device__ __forceinline__ int pages_seen(const CacheParams& p, int b, int t) {
  return (int)(((unsigned)max(keys_seen(p, b, t), 0) + p.page - 1) / p.page);
}
// Pages of its sequence.
__device__ __forceinline__ int pages_of(const CacheParams& p, int b) {
  return (int)(((unsigned)__ldg(p.kv_lens + b) + p.page - 1) / p.page);
}
__device__ __forceinline__ int list_pieces(const CacheParams& p, int seen) {
  return max(1, (min(seen, p.list_count) * p.page + kPiece - 1) / kPiece);
}

// Where a warp is in the CTA's run of pieces.  Positions count pieces and, before each unit's, `cost` places
// for starting and ending it, which nobody fills (KIND_PLAIN: none).
template <int KIND>
struct Cursor {
  static constexpr bool LIST = KIND == KIND_LIST;
  int b, h;
  int t, seen;                               // LIST: packed query, the pages it sees
  int cost;
  long long f, ubeg, uend;                   // piece, and the unit's first and last + 1
  __device__ __forceinline__ void settle(const CacheParams& p, long long end) {   // into the unit that holds f
    while (f < end && f >= uend) {
      ubeg = uend;
      if constexpr (KIND != KIND_PLAIN) {
        ubeg += cost;
        f += cost;
      }
      if (++h == p.Hkv) {
        h = 0;
        if constexpr (LIST) {
          ++t;                               // f < end: there is another unit
          while (t >= __ldg(p.cu_q + b + 1)) ++b;
          seen = pages_seen(p, b, t);
          uend = ubeg + list_pieces(p, seen);
        } else {
          int np;
          do np = pieces_of<KIND>(p, ++b);
          while (np == 0);
          uend = ubeg + np;
        }
      } else {
        uend = ubeg + (LIST ? list_pieces(p, seen) : pieces_of<KIND>(p, b));
      }
    }
  }
};

// LIST: attention over listed pages.  p.list [K/V head][query][list_count] holds page numbers within the
// query's sequence; p.rep virtual heads of p.g query heads share a K/V head (p.Hkv counts virtual ones).
template <int D, int KIND>
__global__ void __launch_bounds__(kThreads, 2)
    fwd_cache_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                            const CacheParams p, const int rows_max) {
  using C = DecCfg<D>;
  constexpr bool LIST = KIND == KIND_LIST, SIDE = KIND == KIND_SIDE;
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
  const int seqs = SIDE && p.side == SIDE_BOTH ? p.B + p.two.B : p.B;
  const int per_thread = (seqs + kThreads - 1) / kThreads;
  const int b_lo = min(tid * per_thread, seqs), b_hi = min(b_lo + per_thread, seqs);
  long long mine = 0;
  int units = 0;                             // (per K/V head)
  bool wrong = false;
  for (int b = b_lo; b < b_hi; ++b) {
    if constexpr (SIDE) {
      const PartSeq s(p, b);
      const int c0 = __ldg(s.cu + s.b), n = __ldg(s.cu + s.b + 1) - c0, len = __ldg(s.lens + s.b);
      wrong |= s.wrong(p, c0, n, len);
      if (n > 0) {
        mine += max(1, (len + kPiece - 1) / kPiece);
        ++units;
      }
      continue;
    }
    const int c0 = __ldg(p.cu_q + b), c1 = __ldg(p.cu_q + b + 1), len = __ldg(p.kv_lens + b), n = c1 - c0;
    wrong |= c0 < 0 || c1 < c0 || n > p.max_q || len < 0 || len > p.max_len || (p.causal && n > len) ||
             (b == 0 && c0 != 0) || (b == p.B - 1 && c1 != p.total_q);
    if (!LIST && n > 0) {
      mine += max(1, (len + kPiece - 1) / kPiece);
      ++units;
    }
  }
  // LIST: thread t adds up queries [t per_query, ...) instead.
  const int per_query = (p.total_q + kThreads - 1) / kThreads;
  const int t_lo = min(tid * per_query, p.total_q), t_hi = min(t_lo + per_query, p.total_q);
  int b_first = 0;
  if constexpr (LIST) {
    if (t_lo < t_hi) b_first = seq_of(p, t_lo);
    int b = b_first;
    for (int t = t_lo; t < t_hi; ++t) {
      while (b < p.B - 1 && t >= __ldg(p.cu_q + b + 1)) ++b;
      mine += list_pieces(p, pages_seen(p, b, t));
    }
    units = t_hi - t_lo;
  }
  // A unit costs as much as kUnitCost pieces, or, with little work, a quarter of a CTA's pieces.
  int cost = 0;
  if constexpr (KIND != KIND_PLAIN) {
    long long all = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (lane == 0) misc[warp] = all;
    __syncthreads();
    all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) all += misc[w];
    cost = (int)min((long long)kUnitCost, all * p.Hkv / gridDim.x / 4);
    mine += (long long)cost * units;
    __syncthreads();                         // misc has been read
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
    if (SIDE && p.side != SIDE_IN && blockIdx.x == 0) *p.side_bad = bad;
  }
  if (bad || (SIDE && p.side == SIDE_IN && *p.side_bad)) return;
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
    int b = LIST ? b_first : b_lo, t = t_lo;
    long long at = before;
    for (;;) {
      if constexpr (LIST) {
        while (t >= __ldg(p.cu_q + b + 1)) ++b;
      }
      const int np = LIST ? list_pieces(p, pages_seen(p, b, t)) : pieces_of<KIND>(p, b);
      const long long step = np > 0 ? (long long)(np + cost) * p.Hkv : 0;
      if (rs < at + step) break;
      at += step;
      if (LIST) ++t;
      else ++b;
    }
    misc[0] = b;
    misc[1] = at;
    if (LIST) misc[2] = t;
  }
  __syncthreads();
  Cursor<KIND> seg;                          // the unit being worked on
  seg.b = (int)misc[0];
  seg.cost = cost;
  seg.t = seg.seen = 0;
  if constexpr (LIST) {
    seg.t = (int)misc[2];
    seg.seen = pages_seen(p, seg.b, seg.t);
  }
  {
    const int np = LIST ? list_pieces(p, seg.seen) : pieces_of<KIND>(p, seg.b);
    seg.h = (int)((rs - misc[1]) / (np + cost));
    seg.ubeg = misc[1] + (long long)seg.h * (np + cost) + cost;
    seg.uend = seg.ubeg + np;
    seg.f = max(rs, seg.ubeg);
  }
  const long long first = seg.f;             // the CTA's first piece

  // ---- this warp's loads, STAGES pieces ahead of its work
  const int page_shift = 31 - __clz(p.page);
  const int grp = lane & 1;                  // half of a piece (16 keys) this lane looks after
  uint8_t* ring = smem + warp * C::STAGES * 2 * C::KB;
  Cursor<KIND> ahead = seg;
  ahead.f = first + warp;
  ahead.settle(p, re);
  const int kv_heads = LIST ? p.Hkv / p.rep : p.Hkv;
  auto kv_head = [&](int h) -> int { return LIST && p.rep > 1 ? h / p.rep : h; };
  int key_ahead = 0;                         // LIST: the first key of this lane's half of the piece at `ahead`
  // The page of this lane's half of the piece at `ahead`: -1 behind the last key, -2 bad.
  auto page_at = [&]() -> int {
    if (ahead.f >= re) return -1;
    int key = (int)(ahead.f - ahead.ubeg) * kPiece + grp * 16;
    if constexpr (LIST) {
      const int e = key >> page_shift;
      if (e >= min(ahead.seen, p.list_count)) return -1;
      const int lp = __ldg(p.list + ((long long)kv_head(ahead.h) * p.total_q + ahead.t) * p.list_count + e);
      if (lp < 0) return -1;
      if (lp >= ahead.seen) {                // a page that the query does not see (later ones of its sequence may)
        if (lp < pages_of(p, ahead.b)) return -1;
        atomicExch(p.status, DEV_BAD_PAGE);
        return -2;
      }
      key = key_ahead = (lp << page_shift) + (key & (p.page - 1));
    } else if constexpr (SIDE) {
      if (key >= __ldg(PartSeq(p, ahead.b).lens + PartSeq(p, ahead.b).b)) return -1;
    } else {
      if (key >= __ldg(p.kv_lens + ahead.b)) return -1;
    }
    const int* table = p.table + (long long)ahead.b * p.max_pages;
    if constexpr (SIDE) table = PartSeq(p, ahead.b).table + (long long)PartSeq(p, ahead.b).b * PartSeq(p, ahead.b).max_pages;
    const int pg = __ldg(table + (key >> page_shift));
    if (pg < 0 || pg >= p.num_pages) {
      atomicExch(p.status, DEV_BAD_PAGE);
      return -2;
    }
    return pg;
  };
  // Scale of this lane's half: K for lanes with bit 1 clear, V with it set.
  auto scale_of = [&](int pg, int h) -> float {
    return pg >= 0 ? __ldg(((lane & 2) ? p.v_scale : p.k_scale) + (long long)pg * kv_heads + h) : 0.f;
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
      const int z = pg * kv_heads + kv_head(ahead.h);
      const uint32_t dst = smem_u32(ring + stage * 2 * C::KB) + lane * box;
      tma_load_3d(dst, &tm_k, 0, line, z, bar);
      tma_load_3d(dst + C::KB, &tm_v, 0, line, z, bar);
    }
  };
  int pages[C::STAGES + 1], heads[C::STAGES + 1];     // of the pieces under way, oldest first; one more looked up
  int keys[LIST ? C::STAGES + 1 : 1];                 // LIST: first key of this lane's half of each
  bool ok = true;
#pragma unroll
  for (int i = 0; i <= C::STAGES; ++i) {
    pages[i] = page_at();
    heads[i] = kv_head(ahead.h);
    if (LIST) keys[i] = key_ahead;
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
  long long f = first + warp;                // this warp's next piece

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
    int q0, n, len, causal = p.causal;
    if constexpr (SIDE) {
      const PartSeq s(p, seg.b);
      q0 = __ldg(s.cu + s.b);
      n = __ldg(s.cu + s.b + 1) - q0;
      len = __ldg(s.lens + s.b);
      causal = s.causal;
    } else {
      q0 = LIST ? seg.t : __ldg(p.cu_q + seg.b);
      n = LIST ? 1 : __ldg(p.cu_q + seg.b + 1) - q0;
      len = LIST ? keys_seen(p, seg.b, seg.t) : __ldg(p.kv_lens + seg.b);
    }
    const int part_of_keys = SIDE && seg.b >= p.B ? 1 : 0;
    if (LIST && seg.f == seg.ubeg) {         // entries behind as many as the query sees pages are not read: none may count
      const int* entries = p.list + ((long long)kv_head(seg.h) * p.total_q + seg.t) * p.list_count;
      for (int e = seg.seen + tid; e < p.list_count; e += kThreads) {
        const int lp = __ldg(entries + e);
        if (lp >= 0 && (lp < seg.seen || lp >= pages_of(p, seg.b))) atomicExch(p.status, DEV_BAD_PAGE);
      }
    }
    const long long send = min(seg.uend, re);
    const int rows = n * g;
    // Visible keys of this thread's two rows.
    int lim[2];
    float crow[2];
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = rq + 8 * i, qi = r / g;
      lim[i] = causal && r < rows ? len - n + qi + 1 : len;
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
    const int min_lim = causal ? len - n + 1 : len;
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
        // First key of each half (LIST: on pages of their own).
        const int kh[2] = {LIST ? __shfl_sync(0xffffffffu, keys[0], 0) : key0,
                           LIST ? __shfl_sync(0xffffffffu, keys[0], 1) - 16 : key0};
        const bool partial = (LIST ? max(kh[0], kh[1]) : key0) + kPiece > min_lim || !got0 || !got1;
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
          const int key = key0 + lane;       // (LIST: all rows see the same keys)
          if (!LIST && key >= min_lim && key < len && (lane < 16 ? got0 : got1)) {
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
              if (kh[nb >> 1] + key_of(nb, i & 1) >= lim[i >> 1] || !((nb >> 1) ? got1 : got0)) s[nb][i] = -INFINITY;
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
            live[x] = kh[t] + key_of(2 * t + (x >> 1), x & 1) < len && (t ? got1 : got0);
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
        if (LIST) keys[i] = keys[i + 1];
      }
      ahead.f += kWarps;
      ahead.settle(p, re);
      pages[C::STAGES] = page_at();
      heads[C::STAGES] = kv_head(ahead.h);
      if (LIST) keys[C::STAGES] = key_ahead;
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
        *rec = make_int4(seg.h | part_of_keys << 30, q0, n, 2 * ((int)((seg.uend - 1) / run) - (int)blockIdx.x) + second);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = rq + 8 * i, qi = r / g;
        if (r >= rows) continue;
        // Columns of o[j][2i] and o[j][2i + 1]: for d = 128, 32 c + j and 32 c + 16 + j; d = 64, 16 c + j and 16 c + 8 + j.
        if (whole) {
          float inv = l[i] == 0.f ? 0.f : rref / l[i];
          float lse2 = m[i] - kShift + __log2f(l[i]);
          const long long row = (long long)(seg.h * g + (r - qi * g)) * p.total_q + q0 + qi;
          if constexpr (SIDE) {              // columns 8 k .. 8 k + 7 of each half: two pieces of 4
            const long long pieces = (long long)p.total_q * g;     // from one piece of the row to the next
            float4* side = side_piece<D>(p, part_of_keys, seg.h, q0, r, c * (D / 16));
            float2 w = make_float2(1.f, 0.f);
            if (p.side == SIDE_IN) w = join_side(p, side_row(p, seg.h, q0, r), lse2, lse2);
            inv *= w.x;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int k = 0; k < C::NACC / 4; ++k) {
                float4 y = make_float4(o[4 * k][2 * i + e] * inv, o[4 * k + 1][2 * i + e] * inv, o[4 * k + 2][2 * i + e] * inv,
                                       o[4 * k + 3][2 * i + e] * inv);
                float4* at = side + (e * (C::NACC / 4) + k) * pieces;
                if (p.side != SIDE_IN) {
                  *at = y;
                  continue;
                }
                const float4 x = *at;
                o[4 * k][2 * i + e] = y.x + w.y * x.x;
                o[4 * k + 1][2 * i + e] = y.y + w.y * x.y;
                o[4 * k + 2][2 * i + e] = y.z + w.y * x.z;
                o[4 * k + 3][2 * i + e] = y.w + w.y * x.w;
              }
            if (p.side != SIDE_IN) {
              if (c == 0) p.side_lse[part_of_keys][side_row(p, seg.h, q0, r)] = lse2;
              continue;
            }
            inv = 1.f;
          }
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
          if (c == 0) p.lse[row] = lse2 * kLn2;
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
    if (KIND != KIND_PLAIN && send == seg.uend && send < re) f += cost;      // on to the next unit
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
template <int D, int CPT, int JOIN, bool COMPACT, bool SIDE>
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
    int4 rec = recs[cta];
    const int part_of_keys = SIDE ? rec.x >> 30 : 0;
    if (SIDE) rec.x &= (1 << 30) - 1;
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
    float inv = l == 0.f ? 0.f : ref / l, lse2 = m + __log2f(l);
    if constexpr (SIDE) {
      const long long pieces = (long long)p.total_q * p.g;         // from one piece of the row to the next
      float4* side = side_piece<D>(p, part_of_keys, rec.x, rec.y, r, cg * CPT);
      float2 w = make_float2(1.f, 0.f);
      if (p.side == SIDE_IN) w = join_side(p, side_row(p, rec.x, rec.y, r), lse2, lse2);
      inv *= w.x;
#pragma unroll
      for (int c = 0; c < CPT; ++c) {
        o[c] = make_float4(o[c].x * inv, o[c].y * inv, o[c].z * inv, o[c].w * inv);
        if (p.side != SIDE_IN) {
          side[c * pieces] = o[c];
          continue;
        }
        const float4 x = side[c * pieces];
        o[c] = make_float4(o[c].x + w.y * x.x, o[c].y + w.y * x.y, o[c].z + w.y * x.z, o[c].w + w.y * x.w);
      }
      if (p.side != SIDE_IN) {
        if (cg == 0) p.side_lse[part_of_keys][side_row(p, rec.x, rec.y, r)] = lse2;
        continue;
      }
      inv = 1.f;
    }
    uint32_t y[2 * CPT];
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      y[2 * c] = pack_bf16x2(o[c].x * inv, o[c].y * inv);
      y[2 * c + 1] = pack_bf16x2(o[c].z * inv, o[c].w * inv);
    }
    uint16_t* out = static_cast<uint16_t*>(p.o) + row * D + cg * CPT * 4;
    if constexpr (CPT == 1) *reinterpret_cast<uint2*>(out) = make_uint2(y[0], y[1]);
    else *reinterpret_cast<uint4*>(out) = make_uint4(y[0], y[1], y[2], y[3]);
    if (cg == 0) p.lse[row] = lse2 * kLn2;
  }
}

// Both parts of each row joined.  Block: 256 rows of a K/V head and two pieces of 4 columns, a row per thread, so that
// neighbours read side by side.
template <int D>
__global__ void __launch_bounds__(256) fwd_cache_join_kernel(const CacheParams p, const int chunks) {
  pdl_wait();
  pdl_trigger();
  if (*p.side_bad) return;
  const long long rows = (long long)p.total_q * p.g;
  const int u = blockIdx.x / chunks, h = u / (D / 8), pair = u - h * (D / 8);
  const long long r = (long long)(blockIdx.x - u * chunks) * 256 + threadIdx.x;
  if (r >= rows) return;
  const long long at = 2LL * u * rows + r;             // piece h D / 4 + 2 pair
  const float4* a = reinterpret_cast<const float4*>(p.side_o[0]) + at;
  const float4* b = reinterpret_cast<const float4*>(p.side_o[1]) + at;
  const float4 a0 = a[0], a1 = a[rows], b0 = b[0], b1 = b[rows];
  float joint;
  const float2 w = join_two(p.side_lse[1][h * rows + r], p.side_lse[0][h * rows + r], joint);
  const long long t = r / p.g, row = ((long long)h * p.g + (r - t * p.g)) * p.total_q + t;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + row * D + pair * 8) = make_uint4(
      pack_bf16x2(b0.x * w.x + a0.x * w.y, b0.y * w.x + a0.y * w.y), pack_bf16x2(b0.z * w.x + a0.z * w.y, b0.w * w.x + a0.w * w.y),
      pack_bf16x2(b1.x * w.x + a1.x * w.y, b1.y * w.x + a1.y * w.y), pack_bf16x2(b1.z * w.x + a1.z * w.y, b1.w * w.x + a1.w * w.y));
  if (pair == 0) p.lse[row] = joint * kLn2;
}

template <int D, int KIND>
cudaError_t launch_decode(const CacheMaps& maps, const CacheParams& p, int rows, int grid, cudaStream_t s) {
  using C = DecCfg<D>;
  static std::once_flag flags[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::call_once(flags[dev & 63], [&] {
    attr_err[dev & 63] = cudaFuncSetAttribute(fwd_cache_decode_kernel<D, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (attr_err[dev & 63] != cudaSuccess) return attr_err[dev & 63];
  // A dependent launch of whatever runs before: the kernel waits for it to be done, but is in place by then.
  e = launch_pdl(fwd_cache_decode_kernel<D, KIND>, dim3(grid), dim3(kThreads), C::SMEM, s, maps.k, maps.v, p, rows);
  if (e != cudaSuccess) return e;
  return launch_fwd_cache_merge(p, D, rows, grid, s);
}

}  // namespace

cudaError_t launch_fwd_cache_merge(const CacheParams& p, int d, int rows, int ctas, cudaStream_t s) {
  int shift = 0;
  const int max_q = p.side == SIDE_BOTH && p.two.max_q > p.max_q ? p.two.max_q : p.max_q;
  while ((1 << shift) < rows && (1 << shift) < (long long)max_q * p.g) ++shift;       // rows in use
  auto go = [&](auto kernel, int cpt, bool compact) {
    const int shares = (((d / 4 / cpt) << shift) + 127) / 128;
    const int blocks = compact ? 4 * kSMs : ctas * shares;
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(128), 0, s, p, rows, shift, ctas);
  };
  // Few units of many partials each: latency again (a sequence of 30000 keys, 32 rows: 33 us against 35).
  const long long units = ((long long)p.B + (p.side == SIDE_BOTH ? p.two.B : 0)) * p.Hkv * (((long long)max_q * p.g + rows - 1) / rows);
  auto pick = [&](auto dim, auto side) {
    constexpr int D = dim;
    constexpr bool S = side;
    if (rows <= kCacheDecodeRows || units * 4 <= ctas) {
      if (((d / 4) << shift) / 128 * ctas > 16 * kSMs && ctas <= 1024) return go(fwd_cache_merge_kernel<D, 1, 8, true, S>, 1, true);
      return go(fwd_cache_merge_kernel<D, 1, 8, false, S>, 1, false);
    }
    return go(fwd_cache_merge_kernel<D, 2, 2, false, S>, 2, false);
  };
  using I64 = std::integral_constant<int, 64>;
  using I128 = std::integral_constant<int, 128>;
  if (p.side != SIDE_NONE) return d == 64 ? pick(I64(), std::true_type()) : pick(I128(), std::true_type());
  return d == 64 ? pick(I64(), std::false_type()) : pick(I128(), std::false_type());
}

cudaError_t launch_fwd_cache_join(const CacheParams& p, int d, cudaStream_t s) {
  const long long chunks = ((long long)p.total_q * p.g + 255) / 256, blocks = chunks * p.Hkv * (d / 8);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks);
  return d == 64 ? launch_pdl(fwd_cache_join_kernel<64>, grid, dim3(256), 0, s, p, (int)chunks)
                 : launch_pdl(fwd_cache_join_kernel<128>, grid, dim3(256), 0, s, p, (int)chunks);
}

size_t cache_decode_workspace_bytes(int rows, int d, int sms) { return cache_ws(2 * sms, rows, d).total; }

cudaError_t launch_fwd_cache_decode(const CacheMaps& maps, const CacheParams& p, int d, int sms, cudaStream_t s) {
  const int max_q = p.side == SIDE_BOTH && p.two.max_q > p.max_q ? p.two.max_q : p.max_q;
  const int rows = max_q * p.g, grid = 2 * sms;        // as in the workspace's size
  if (p.side != SIDE_NONE)
    return d == 64 ? launch_decode<64, KIND_SIDE>(maps, p, rows, grid, s) : launch_decode<128, KIND_SIDE>(maps, p, rows, grid, s);
  return d == 64 ? launch_decode<64, KIND_PLAIN>(maps, p, rows, grid, s) : launch_decode<128, KIND_PLAIN>(maps, p, rows, grid, s);
}

cudaError_t launch_fwd_cache_pages(const CacheMaps& maps, const CacheParams& p, int d, int sms, cudaStream_t s) {
  const int grid = 2 * sms;
  return d == 64 ? launch_decode<64, KIND_LIST>(maps, p, p.g, grid, s) : launch_decode<128, KIND_LIST>(maps, p, p.g, grid, s);
}

}  // namespace attn
