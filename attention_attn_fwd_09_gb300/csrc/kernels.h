// Launch interfaces shared between the host entry points (api.cu) and the kernel
// translation units.  Host-only types; no torch.
#pragma once
#include <cstddef>
#include <cstdint>
#include <utility>
#include <cuda.h>
#include <cuda_runtime.h>

namespace attn {

// Launches `kernel` as a programmatic dependent of the stream's previous kernel: its CTAs
// may be scheduled once every CTA of that kernel has called pdl_trigger (or exited), and
// they must call pdl_wait before touching anything the previous kernel writes.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Device status word codes (see attn_device_status).  Kernels never trap: a kernel that
// gives up on a bounded wait, or finds its device-side arguments invalid, writes one of
// these and returns.
enum : int { DEV_OK = 0, DEV_TIMEOUT = 1, DEV_BAD_OFFSETS = 2, DEV_BAD_PAGE = 3 };

struct FwdParams {
  int B, Hq, Hkv, N, g;      // N: query length
  int Nk, koff;              // key length and Nk - N (query i stands at key position i + koff)
  int causal;
  int pair_heads;          // 1: a CTA's two tiles are query heads 2p, 2p+1 of one KV group
  int n_qblk, n_kvblk;     // ceil(N / 128), ceil(Nk / 128)
  int units_per_row;       // CTAs per query-row slot (see fwd.cu unit mapping)
  int n_rowslots;          // query-row slots per head (pair) sequence
  int split_from;          // units >= split_from run as two one-tile CTAs (the last, partial wave)
  int prefetch_ahead;      // > 0: a CTA prefetches into L2 the first tiles of CTA blockIdx + this
  // Grouped decode mode (queries after a key cache, g * N <= 128): one CTA per (K/V head,
  // key split) with one tile holding the group's g query heads x N queries; each CTA writes
  // a normalised partial O and LSE for its key range, merged by launch_fwd_merge.
  int pack;                // 0 ordinary, 1 grouped decode, 2 packed variable-length sequences
  int kv_splits, blocks_per_split;
  unsigned q_tile_bytes;   // bytes one Q tile load delivers (a full tile, or g * N rows of it)
  float* part_o;           // [kv_splits][B * Hkv][128][D] fp32
  float* part_lse;         // [kv_splits][B * Hkv][128] fp32, natural log
  // Packed variable-length mode (pack == 2): Q/O [Hq, N, D], K/V [Hkv, Nk, D] with N and Nk
  // the packed lengths; each CTA takes one record of the unit table written by
  // launch_varlen_schedule (CTAs past *vl_count have no record and exit at once).
  const int* cu_q;         // [B + 1] query row offsets (device)
  const int* cu_k;         // [B + 1] key row offsets (device)
  const int* vl_count;     // records in the table
  const int4* vl_units;    // {b, hq0 | hq1 << 16, r0, r1}: rows r0, r1 of sequence b (r1 < 0: one tile)
  void* o_ptr;             // O, for tiles that end inside their sequence (plain stores)
  float c;                 // scale * log2(e)
  float tau;               // conditional-rescale threshold, log2 units
  float* lse;              // [B, Hq, N] fp32, natural log
  unsigned long long wait_ns;
  int* status;
  unsigned long long* rescale_count;  // optional counter (nullptr = off)
  int test_skip_first_kv;             // test hook: never load ring index 0 (exercises timeouts)
};

struct FwdMaps {
  CUtensorMap q, k, v, o;
};

// Forward: D in {64, 128}; poly_per_16 in {0, 4, 16} elements of every 16 computed by
// the FMA polynomial instead of MUFU.EX2.
cudaError_t launch_fwd(const FwdMaps& maps, const FwdParams& p, int D, int poly_per_16, int grid,
                       cudaStream_t stream);
// Grouped decode mode: combine the kv_splits partial results into o [B,Hq,N,D] bf16 and
// lse [B,Hq,N] fp32.
cudaError_t launch_fwd_merge(const FwdParams& p, int D, void* o, cudaStream_t stream);

// Packed variable-length mode: the unit table.  One CTA validates the offsets and writes
// one record per CTA, longest sequence first: for the forward two 128-row query tiles of
// one sequence, for the backward one 128-key block of one sequence and K/V head.
struct VarlenSched {
  const int* cu_q;
  const int* cu_k;
  int backward;            // 0: forward records; 1: backward records {b, hkv, key block, 0}
  int single;              // forward: one query tile per record (the one-tile kernel, d > 128)
  int B, Hq, Hkv, pair_heads, causal, total_q, total_k;
  int nbins;               // work classes (a sequence's key blocks, clamped to nbins - 1)
  int cap;                 // records the table can hold
  int lpt;                 // 1: longest first; 0: every record in one class (arrival order)
  int* header;             // [0] records written; [1] 0, or 1 when the offsets were invalid
  int4* units;             // [cap] records
  int* status;             // device status word (DEV_BAD_OFFSETS on invalid offsets)
};
cudaError_t launch_varlen_schedule(const VarlenSched& s, cudaStream_t stream);
size_t fwd_smem_bytes(int D);
// Persistent two-tile forward (fwd_persist.cu), d = 64 or 128, ordinary mode, MUFU
// exponentials: grid CTAs walk entries 0 .. n_entries - 1 of the work list (units below
// p.split_from whole, then one-tile halves) in steps of grid; O is written through p.o_ptr.
cudaError_t launch_fwd_persistent(const FwdMaps& maps, const FwdParams& p, int D, int grid, int n_entries,
                                  cudaStream_t stream);
// One-tile forward (fwd_wide.cu) for d = 128, 192 or 256: one 128-row query tile per CTA,
// grid = B * Hq * ceil(N / 128); same parameters as launch_fwd.  pack == 1 (grouped decode,
// d = 128: grid = B * Hkv * kv_splits, then launch_fwd_merge) and pack == 2 (packed
// sequences, d = 192, 256: grid = the table's bound) as for launch_fwd.
cudaError_t launch_fwd_wide(const FwdMaps& maps, const FwdParams& p, int D, int grid, cudaStream_t stream);

// FP8 forward (fwd_fp8.cu), d = 128, ordinary tiling: Q/K/V maps over e4m3 bytes (boxes
// of 128 rows x 128 bytes), O map as for launch_fwd; block scales per 128 rows of a head.
struct Fp8Scales {
  const float* q;   // [B, Hq, ceil(N / 128)]
  const float* k;   // [B, Hkv, ceil(N / 128)]
  const float* v;   // [B, Hkv, ceil(N / 128)]
};
cudaError_t launch_fwd_fp8(const FwdMaps& maps, const FwdParams& p, const Fp8Scales& sc, int grid, cudaStream_t stream);
size_t fwd_fp8_smem_bytes();
// Block quantiser: x bf16 [heads, N, 128] -> x8 e4m3 [heads, N, 128], scales [heads, ceil(N / 128)].
cudaError_t launch_quantize_fp8(const void* x, void* x8, float* scales, long long heads, int N, cudaStream_t stream);

// Software exp2 accuracy / throughput test entry: variant 0 = production polynomial,
// 1 = full-range polynomial, 2 = MUFU ex2.approx.
cudaError_t launch_exp2_test(const float* x, float* y, long long n, int variant, cudaStream_t s);

// Backward.
struct BwdParams {
  int B, Hq, Hkv, N, g, D;
  int causal, deterministic;
  float scale, c;            // softmax scale; scale * log2(e)
  const void *q, *k, *v, *o, *dout;
  const float* lse;
  void *dq, *dk, *dv;
  float* dq_acc;             // [B, Hq, ceil(N/128)*128, D] fp32 workspace (rows padded to whole tiles)
  float* delta;              // [B, Hq, N] fp32 workspace (rowsum(dO o O))
  float* lse2;               // [B, Hq, N] fp32 workspace (LSE * log2 e)
  int* sem;                  // deterministic-order counters
  float* dq_acc2;            // deterministic, d <= 128, not packed: the second accumulator
                             // (shaped as dq_acc); null otherwise
  unsigned long long wait_ns;
  int* status;
  // Packed sequences (varlen = 1): N is total_q, Q/O/dO/dQ [Hq, total_q, D], K/V/dK/dV
  // [Hkv, total_k, D]; dq_acc is [Hq, total_q + 128 B, D] with sequence b's rows starting
  // at cu_q[b] + 128 b (room for its last tile's padding), sem [Hq][sem_stride].
  int varlen, total_k, sem_stride;
  const int* cu_q;
  const int* cu_k;
  const int* vl_count;
  const int4* vl_units;      // {b, hkv, key block n, 0}
};
struct BwdMaps {
  CUtensorMap q, k, v, dout, dk, dv;
};
cudaError_t launch_bwd(const BwdMaps& maps, const BwdParams& p, cudaStream_t stream);
size_t bwd_workspace_bytes(int B, int Hq, int Hkv, int N, int d, int deterministic);
// Packed sequences: workspace layout (dq_acc, delta, lse2, sem, then the unit table).
struct BwdVarlenLayout {
  size_t dq_acc, delta, lse2, sem, table, total;
  long long rows_pad, cap;
  int sem_stride;
};
BwdVarlenLayout bwd_varlen_layout(int B, int Hq, int Hkv, int total_q, int total_k, int d, int deterministic);
// Points p->dq_acc, delta, lse2, sem (and, deterministic, dq_acc2) into the caller's
// workspace.
void bwd_workspace_carve(void* ws, int B, int Hq, int Hkv, int N, int d, int deterministic, BwdParams* p);
// Backward for d = 192, 256 (bwd_wide.cu): maps as launch_bwd except q and dout, whose
// boxes are 64 rows; workspace: dQacc [B, Hq, ceil(N/64)*64, d], D and LSE2 [B, Hq, N],
// counters [B, Hq, ceil(N/64), 2] when deterministic.
size_t bwd_wide_workspace_bytes(int B, int Hq, int N, int d, int deterministic);
void bwd_wide_workspace_carve(void* ws, int B, int Hq, int N, int d, int deterministic, BwdParams* p);
cudaError_t launch_bwd_wide(const BwdMaps& maps, const BwdParams& p, cudaStream_t stream);

// Rotary positions (rope.cu).  Element strides of batch, head and token; columns contiguous.
struct RopeTensor {
  const void* in;
  void* out;
  long long in_b, in_h, in_n, out_b, out_h, out_n;
};
struct RopeParams {
  RopeTensor q, k;           // k unused when Hk = 0
  const double* inv_freq;    // [rot / 2] radians per position (device)
  const int* positions;      // [B, N] (device) or null: 0 .. N - 1
  int B, N, Hq, Hk, d, rot;
  float mscale, sign;        // factor on the rotated part; +1 forward, -1 transposed
  int tile_shift, tiles, head_group;   // filled in by launch_rope: log2(tokens per CTA), tiles per sequence, heads per CTA
  // Not null: packed rows (B = 1; d = 64 or 128) that end their sequences, which gives their positions where
  // positions is null (offsets [seqs + 1], lengths [seqs]); the launch runs beside the kernel before it in the
  // stream, which calls pdl_trigger and whose outputs it does not touch.
  const int *cu, *kv_lens;
  int seqs;
};
// vec: elements per access (8, 4 or 1) that every pointer, stride and rot allow.
cudaError_t launch_rope(RopeParams p, int vec, int interleaved, int sms, cudaStream_t s);

// Rows into the paged e4m3 cache (kv_append.cu); d = 64 or 128, page = 16, 32, 64 or 128.
struct AppendParams {
  const void *k, *v;         // bf16 [Hkv, total, d], strides in elements, columns contiguous
  long long k_h, k_t, v_h, v_t;
  void *k_cache, *v_cache;   // [num_pages, Hkv, page, d] e4m3
  float *k_scale, *v_scale;  // [num_pages, Hkv]
  const int *table, *cu, *kv_lens;   // [B, max_pages], [B + 1], [B]
  int B, Hkv, total, num_pages, page, max_pages, max_len;
  int page_shift;            // log2(page), filled in by launch_kv_append
  int* status;
};
cudaError_t launch_kv_append(AppendParams p, int d, int sms, cudaStream_t s);

// The same with K rotated on the way and bounds of each page's K codes (rope_append.cu).
struct RopeAppendParams {
  AppendParams a;
  const double* inv_freq;    // [rot / 2] radians per position (device); rot = 0: K as it is
  const int* positions;      // [total] (device) or null: the rows' places in their sequences
  int rot, interleaved;
  float mscale;
  uint8_t* bounds;           // [num_pages, Hkv, 2, d] smallest and largest code per column, or null
  const void* q;             // bf16 [Hq, total, d], element strides of head and row; rows on 16 bytes, rot a multiple of 8
  void* q_out;
  long long q_h, q_t, o_h, o_t;
  int Hq;
  int heads_per_cta, slots;  // filled in by launch_rope_append
};
// *queries in: whether q may rotate in the same launch; out: whether it does.
cudaError_t launch_rope_append(RopeAppendParams p, int d, int sms, bool* queries, cudaStream_t s);

// Choice of pages by their bounds (select_pages.cu); d = 64 or 128.
struct SelectParams {
  const void* q;             // bf16 [Hq, total_q, d]
  const uint8_t* bounds;     // [num_pages, Hkv, 2, d]
  const float* k_scale;      // [num_pages, Hkv]
  const int *table, *cu_q, *kv_lens;
  int* out;                  // [Hkv, total_q, count]
  int B, Hkv, g, total_q, max_q, num_pages, page, max_pages, max_len, count, first, last, causal;
  float *scores, *errors;    // workspace, see select_ws
  unsigned long long* exact;
  int* near;
  int* status;
  int page_shift, qn, groups;   // filled in by launch_select_pages
};
struct SelectWs {
  size_t exact, near, errors, total;   // scores come first
};
SelectWs select_ws(int Hkv, int total_q, int max_pages);
cudaError_t launch_select_pages(SelectParams p, int d, int sms, cudaStream_t s);

// Packed queries over the paged e4m3 cache (fwd_cache.cu).
struct CacheParams {
  const void* q;             // bf16 [Hq, total_q, d]
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int *table, *cu_q, *kv_lens;
  void* o;                   // bf16 [Hq, total_q, d]
  float* lse;                // [Hq, total_q], natural log
  int B, Hq, Hkv, g, total_q, max_q, num_pages, page, max_pages, max_len;   // max_len = max_pages * page
  int causal;
  float c;                   // scale * log2(e)
  void* ws;
  unsigned long long wait_ns;
  int* status;
  int test_skip_first_kv;    // test hook: each CTA never issues its first K copy
  // Listed pages (launch_fwd_cache_pages): page numbers within each query's sequence, [K/V heads][total_q]
  // [list_count], negative ones left out; g, Hkv count virtual heads, rep of which share a K/V head.
  const int* list;
  int list_count, rep;
  // Keys in two parts (a shared prefix, then a sequence's own).  A part's result goes to its side_o
  // [Hkv][d / 4][total_q g] (pieces of 4 columns; a K/V head's rows are query by query, its heads side by side) and
  // side_lse [Hkv][total_q g] (log2) instead of o and lse.  One launch may do both parts (SIDE_BOTH: `two` is the second
  // one, launch_fwd_cache_join joins them), or one the first part (SIDE_OUT) and another the second, joining it with
  // the first's results (SIDE_IN).
  int side;
  float *side_o[2], *side_lse[2];
  int* side_bad;             // some offsets were invalid: what comes after writes nothing
  struct {
    const int *table, *cu_q, *kv_lens;
    int B, max_q, max_pages, max_len, causal;
  } two;
};
enum : int { SIDE_NONE = 0, SIDE_OUT = 1, SIDE_IN = 2, SIDE_BOTH = 3 };
// Tensor maps over the codes as 128-byte lines, [num_pages * Hkv][page * d / 128][128], boxes of
// 32 keys (a page of 16: 16 keys), 128-byte swizzle.
struct CacheMaps {
  CUtensorMap k, v;
};
// At most 16 rows (queries x heads of a group) per sequence and K/V head: fwd_cache.cu.  (16 rows, 16
// sequences of 16000 keys: 96 us, the tiles 146; one of 4000: 15.0 against 16.3.)
constexpr int kCacheDecodeRows = 16;
size_t cache_decode_workspace_bytes(int rows, int d, int sms);
// Joins what the main kernel's ctas CTAs left of units cut between them, a dependent launch.
cudaError_t launch_fwd_cache_merge(const CacheParams& p, int d, int rows, int ctas, cudaStream_t s);
cudaError_t launch_fwd_cache_decode(const CacheMaps& maps, const CacheParams& p, int d, int sms, cudaStream_t s);
// Every query by itself, over its list of pages (max_q = 1, g up to kCacheDecodeRows).
cudaError_t launch_fwd_cache_pages(const CacheMaps& maps, const CacheParams& p, int d, int sms, cudaStream_t s);
// More rows: fwd_cache_tile.cu.  Maps as above, but boxes of 128 keys (a smaller page: its keys), and
// K's lines are keys (d bytes; 64-byte swizzle for d = 64).  g <= 256.
size_t cache_tile_workspace_bytes(int d, int sms);
cudaError_t launch_fwd_cache_tile(const CacheMaps& maps, const CacheParams& p, int d, int sms, cudaStream_t s);
cudaError_t launch_fwd_cache_tile_side(const CacheMaps& maps, const CacheParams& p, int d, int sms, cudaStream_t s);
// Both parts' results into o and lse, a dependent launch.
cudaError_t launch_fwd_cache_join(const CacheParams& p, int d, cudaStream_t s);

}  // namespace attn
