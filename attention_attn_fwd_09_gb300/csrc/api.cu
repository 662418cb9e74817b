// C-ABI entry points (declared in include/attn.h): argument checks, TMA tensor maps,
// kernel selection and launch.  No allocation on any call path; every launch goes on
// the caller's stream.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/attn.h"
#include "kernels.h"

namespace attn {

// Status word written by kernels that give up on a bounded wait, and the optional
// rescale counter.  One copy per device; the host reaches them through their device
// addresses (cudaGetSymbolAddress, cached per device).
__device__ int g_dev_status;
__device__ unsigned long long g_rescale_count;

namespace {

thread_local char t_err[512] = "";

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(t_err, sizeof t_err, fmt, ap);
  va_end(ap);
  return code;
}

int cuda_fail(cudaError_t e, const char* where) {
  return fail(ATTN_ERR_CUDA, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
}

std::atomic<float> g_tau{8.0f};
std::atomic<int> g_poly{0};
std::atomic<long long> g_wait_ns{2000000000LL};
std::atomic<int> g_sync_check{0};
std::atomic<int> g_count_rescales{0};
std::atomic<int> g_test_skip_kv{0};
std::atomic<int> g_varlen_lpt{1};
std::atomic<int> g_one_tile_d128{0};
std::atomic<int> g_persistent{0};
std::atomic<int> g_decode_one_tile{1};    // grouped decode at d = 128 through the one-tile kernel (fwd_wide.cu)
std::atomic<int> g_bwd_tile_rows{128};   // d <= 128 backward: 128-row (bwd.cu) or 64-row (bwd_wide.cu) query tiles

struct DevSyms {
  int* status = nullptr;
  unsigned long long* rescale = nullptr;
  int sms = 0;
  cudaError_t err = cudaSuccess;
};
constexpr int kMaxDev = 64;
DevSyms g_syms[kMaxDev];
std::once_flag g_syms_once[kMaxDev];

const DevSyms* dev_syms(int* dev_out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) {
    static DevSyms bad;
    bad.err = e;
    return &bad;
  }
  if (dev_out) *dev_out = dev;
  DevSyms& s = g_syms[dev % kMaxDev];
  std::call_once(g_syms_once[dev % kMaxDev], [&] {
    void* p = nullptr;
    s.err = cudaGetSymbolAddress(&p, g_dev_status);
    s.status = static_cast<int*>(p);
    if (s.err == cudaSuccess) {
      s.err = cudaGetSymbolAddress(&p, g_rescale_count);
      s.rescale = static_cast<unsigned long long*>(p);
    }
    if (s.err == cudaSuccess) s.err = cudaDeviceGetAttribute(&s.sms, cudaDevAttrMultiProcessorCount, dev);
  });
  return &s;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link-time
// dependency on libcuda).
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn g_encode = nullptr;
std::once_flag g_encode_once;
cudaError_t g_encode_err = cudaSuccess;

EncodeFn get_encode() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q{};
    g_encode_err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (g_encode_err == cudaSuccess && q == cudaDriverEntryPointSuccess) g_encode = reinterpret_cast<EncodeFn>(fn);
  });
  return g_encode;
}

// [BH, rows, d] bf16 tensor, boxes of 128 rows x 64 columns, 128-byte swizzle.
// box_rows x box_planes: 128 x 1 for ordinary tiles; N x g to gather the g query heads of
// a group (rows h * N + q) into one tile in grouped decode mode.
int make_map(CUtensorMap* m, const void* base, int d, int rows, long long bh, const char* name, int box_rows = 128,
             int box_planes = 1) {
  EncodeFn enc = get_encode();
  if (!enc) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled unavailable (%s)", cudaGetErrorString(g_encode_err));
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)bh};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)rows * (cuuint64_t)d * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_planes};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(ATTN_ERR_CUDA, "tensor map for %s: CUresult %d", name, (int)r);
  return ATTN_OK;
}

// [BH, rows, 128] e4m3 tensor (one byte per element), boxes of 128 rows x 128 bytes,
// 128-byte swizzle: one box is a whole 128 x 128 tile.
int make_map_e4m3(CUtensorMap* m, const void* base, int rows, long long bh, const char* name) {
  EncodeFn enc = get_encode();
  if (!enc) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled unavailable (%s)", cudaGetErrorString(g_encode_err));
  cuuint64_t dims[3] = {128, (cuuint64_t)rows, (cuuint64_t)bh};
  cuuint64_t strides[2] = {128, (cuuint64_t)rows * 128};
  cuuint32_t box[3] = {128, 128, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(ATTN_ERR_CUDA, "tensor map for %s: CUresult %d", name, (int)r);
  return ATTN_OK;
}

// Codes of a paged cache as lines of line bytes (128 or 64), boxes of box_lines of them, swizzled.
int make_map_cache(CUtensorMap* m, const void* base, int line, int lines, long long pages, int box_lines,
                   const char* name) {
  EncodeFn enc = get_encode();
  if (!enc) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled unavailable (%s)", cudaGetErrorString(g_encode_err));
  cuuint64_t dims[3] = {(cuuint64_t)line, (cuuint64_t)lines, (cuuint64_t)pages};
  cuuint64_t strides[2] = {(cuuint64_t)line, (cuuint64_t)lines * line};
  cuuint32_t box[3] = {(cuuint32_t)line, (cuuint32_t)box_lines, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, line == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(ATTN_ERR_CUDA, "tensor map for %s: CUresult %d", name, (int)r);
  return ATTN_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// wide: the forward also takes d = 192 and 256 (one-tile kernel, fwd_wide.cu).
int check_shape(int B, int Hq, int Hkv, int N, int d, float scale, bool wide = false) {
  if (B < 0 || N < 0) return fail(ATTN_ERR_INVALID_ARG, "B=%d and N=%d must be >= 0", B, N);
  if (Hq <= 0 || Hkv <= 0) return fail(ATTN_ERR_INVALID_ARG, "Hq=%d and Hkv=%d must be >= 1", Hq, Hkv);
  if (Hq % Hkv != 0) return fail(ATTN_ERR_INVALID_ARG, "Hq=%d is not a multiple of Hkv=%d", Hq, Hkv);
  if (wide && (d == 192 || d == 256)) {
  } else if (d != 64 && d != 128) {
    return fail(ATTN_ERR_UNSUPPORTED, wide ? "head dim d=%d (supported: 64, 128, 192, 256)"
                                           : "head dim d=%d (supported here: 64, 128)", d);
  }
  if (!(scale > 0.0f) || !std::isfinite(scale)) return fail(ATTN_ERR_INVALID_ARG, "scale must be finite and > 0");
  if ((long long)B * Hq > 0x7fffffffLL) return fail(ATTN_ERR_INVALID_ARG, "B*Hq too large");
  return ATTN_OK;
}

// The error a non-zero device status word stands for.
int status_fail(int v) {
  if (v == DEV_BAD_OFFSETS)
    return fail(ATTN_ERR_INVALID_ARG, "packed-sequence offsets failed the device check (device status %d)", v);
  if (v == DEV_BAD_PAGE)
    return fail(ATTN_ERR_INVALID_ARG, "a page table entry in use is outside the cache (device status %d)", v);
  return fail(ATTN_ERR_TIMEOUT, "a kernel gave up on a bounded wait (device status %d)", v);
}

int post_launch(const DevSyms* s, cudaStream_t st) {
  if (!g_sync_check.load()) return ATTN_OK;
  cudaError_t e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "stream synchronize");
  int v = 0;
  e = cudaMemcpy(&v, s->status, sizeof v, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "status read");
  if (v != 0) return status_fail(v);
  return ATTN_OK;
}

}  // namespace

void set_last_error(const char* msg) { snprintf(t_err, sizeof t_err, "%s", msg); }

}  // namespace attn

using namespace attn;

extern "C" {

const char* attn_last_error(void) { return t_err; }

const char* attn_version(void) { return "attn-gb300 0.1 (sm_103a)"; }

int attn_set_debug_knobs(float tau, int poly_per_16, long long wait_limit_ns, int sync_check) {
  if (!(tau >= 0.0f) || !std::isfinite(tau)) return fail(ATTN_ERR_INVALID_ARG, "tau must be finite and >= 0");
  if (poly_per_16 != 0 && poly_per_16 != 4 && poly_per_16 != 16)
    return fail(ATTN_ERR_UNSUPPORTED, "poly_per_16=%d (supported: 0, 4, 16)", poly_per_16);
  if (wait_limit_ns <= 0) return fail(ATTN_ERR_INVALID_ARG, "wait limit must be > 0");
  g_tau.store(tau);
  g_poly.store(poly_per_16);
  g_wait_ns.store(wait_limit_ns);
  g_sync_check.store(sync_check ? 1 : 0);
  return ATTN_OK;
}

int attn_set_test_hooks(int skip_first_kv_load) {
  g_test_skip_kv.store(skip_first_kv_load ? 1 : 0);
  return ATTN_OK;
}

int attn_get_debug_knobs(float* tau, int* poly_per_16, long long* wait_limit_ns, int* sync_check) {
  if (tau) *tau = g_tau.load();
  if (poly_per_16) *poly_per_16 = g_poly.load();
  if (wait_limit_ns) *wait_limit_ns = g_wait_ns.load();
  if (sync_check) *sync_check = g_sync_check.load();
  return ATTN_OK;
}

int attn_device_status(int clear) {
  const DevSyms* s = dev_syms(nullptr);
  if (s->err != cudaSuccess) return cuda_fail(s->err, "device symbols");
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_fail(e, "device synchronize");
  int v = 0;
  e = cudaMemcpy(&v, s->status, sizeof v, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "status read");
  if (clear) {
    const int z = 0;
    e = cudaMemcpy(s->status, &z, sizeof z, cudaMemcpyHostToDevice);
    if (e != cudaSuccess) return cuda_fail(e, "status clear");
  }
  if (v != 0) return status_fail(v);
  return ATTN_OK;
}

int attn_rescale_counter(int enable, unsigned long long* value_out) {
  const DevSyms* s = dev_syms(nullptr);
  if (s->err != cudaSuccess) return cuda_fail(s->err, "device symbols");
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_fail(e, "device synchronize");
  unsigned long long v = 0;
  e = cudaMemcpy(&v, s->rescale, sizeof v, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "counter read");
  if (value_out) *value_out = v;
  const unsigned long long z = 0;
  e = cudaMemcpy(s->rescale, &z, sizeof z, cudaMemcpyHostToDevice);
  if (e != cudaSuccess) return cuda_fail(e, "counter clear");
  g_count_rescales.store(enable ? 1 : 0);
  return ATTN_OK;
}

// Grouped decode plan for N queries after Nk keys: used when a group's g query heads x N
// queries fit one 128-row tile (g >= 2); the keys are split so that the grid about fills
// the GPU once.  pack = 0 means the ordinary path.
struct KvPlan {
  int pack, splits, blocks_per_split;
  size_t ws_bytes;
};
static size_t al256(size_t x) { return (x + 255) & ~size_t(255); }
static KvPlan kv_plan(int B, int Hq, int Hkv, int N, int Nk, int d, int sms) {
  KvPlan k{0, 1, 0, 0};
  const int g = Hq / Hkv;
  if (B <= 0 || N <= 0 || Nk <= 0 || g < 2 || (long long)g * N > 128 || d > 128) return k;
  const int nkv = (Nk + 127) / 128;
  const long long units = (long long)B * Hkv;
  long long sp = std::min<long long>(nkv, std::max<long long>(1, sms / units));
  const int bps = (int)((nkv + sp - 1) / sp);
  sp = (nkv + bps - 1) / bps;   // every split holds at least one key block
  k.pack = 1;
  k.splits = (int)sp;
  k.blocks_per_split = bps;
  k.ws_bytes = al256((size_t)sp * units * 128 * d * 4) + al256((size_t)sp * units * 128 * 4);
  return k;
}

// The forward for N queries against Nk keys (query i at key position i + Nk - N).
static int fwd_impl(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv,
                    int N, int Nk, int d, int causal, float scale, void* workspace, size_t ws_bytes,
                    void* stream) {
  int rc = check_shape(B, Hq, Hkv, N, d, scale, true);
  if (rc != ATTN_OK) return rc;
  if (Nk < 0) return fail(ATTN_ERR_INVALID_ARG, "Nk=%d must be >= 0", Nk);
  if (B == 0 || N == 0) return ATTN_OK;
  if (Nk == 0) return fail(ATTN_ERR_INVALID_ARG, "Nk=0 with N=%d queries: the softmax has no keys", N);
  if (causal && N > Nk)
    return fail(ATTN_ERR_INVALID_ARG, "causal needs N <= Nk (got N=%d, Nk=%d): the first queries would see no key",
                N, Nk);
  if (!q || !k || !v || !o || !lse) return fail(ATTN_ERR_INVALID_ARG, "null tensor pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return fail(ATTN_ERR_MISALIGNED, "q, k, v, o and lse must be 16-byte aligned");
  int dev = 0;
  const DevSyms* s = dev_syms(&dev);
  if (s->err != cudaSuccess) return cuda_fail(s->err, "device setup");
  const KvPlan plan = kv_plan(B, Hq, Hkv, N, Nk, d, std::max(1, s->sms));
  const bool pack = plan.pack && workspace != nullptr && ws_bytes >= plan.ws_bytes && aligned16(workspace);

  FwdMaps maps;
  if (pack) {
    if ((rc = make_map(&maps.q, q, d, N, (long long)B * Hq, "q", N, Hq / Hkv)) != ATTN_OK) return rc;
  } else if ((rc = make_map(&maps.q, q, d, N, (long long)B * Hq, "q")) != ATTN_OK) {
    return rc;
  }
  if ((rc = make_map(&maps.k, k, d, Nk, (long long)B * Hkv, "k")) != ATTN_OK) return rc;
  if ((rc = make_map(&maps.v, v, d, Nk, (long long)B * Hkv, "v")) != ATTN_OK) return rc;
  if ((rc = make_map(&maps.o, o, d, N, (long long)B * Hq, "o")) != ATTN_OK) return rc;

  FwdParams p{};
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.N = N; p.g = Hq / Hkv;
  p.Nk = Nk; p.koff = Nk - N;
  p.causal = causal ? 1 : 0;
  p.pair_heads = (p.g >= 2 && p.g % 2 == 0) ? 1 : 0;
  p.n_qblk = (N + 127) / 128;
  p.n_kvblk = (Nk + 127) / 128;
  p.n_rowslots = p.pair_heads ? p.n_qblk : (p.n_qblk + 1) / 2;
  p.units_per_row = p.pair_heads ? B * (Hq / 2) : B * Hq;
  p.c = scale * 1.4426950408889634f;
  p.tau = g_tau.load();
  p.lse = lse;
  p.wait_ns = (unsigned long long)g_wait_ns.load();
  p.status = s->status;
  p.rescale_count = g_count_rescales.load() ? s->rescale : nullptr;
  p.test_skip_first_kv = g_test_skip_kv.load();
  // Units of two tiles, one CTA each.  When the last wave would hold few units (at most
  // half the SMs) they are split into one-tile CTAs, so that the last wave takes one tile's
  // time instead of two tiles' (non-causal only: causal units come longest first, so the
  // last ones are short already).
  const long long units = (long long)p.n_rowslots * p.units_per_row;
  p.split_from = (int)std::min<long long>(units, 0x7fffffffLL);
  if (!p.causal) {
    const long long sms = std::max(1, s->sms);
    const long long rem = units % sms;
    if (units >= sms && rem > 0 && 2 * rem <= sms) p.split_from = (int)(units - rem);
    else if (units < sms && 2 * units <= sms) p.split_from = 0;
  }
  long long grid = p.split_from + 2 * (units - p.split_from);
  p.prefetch_ahead = std::max(1, s->sms);
  p.q_tile_bytes = (unsigned)((d / 64) * 128 * 128);
  // One query tile per CTA (fwd_wide.cu): always for d > 128, and for d = 128 when chosen.
  const bool wide = d > 128 || (d == 128 && !pack && g_one_tile_d128.load());
  if (wide) grid = (long long)B * Hq * p.n_qblk;
  if (pack) {
    p.pack = 1;
    p.kv_splits = plan.splits;
    p.blocks_per_split = plan.blocks_per_split;
    p.q_tile_bytes = (unsigned)((d / 64) * 128 * N * p.g);   // NCH boxes of 64 columns x N rows x g heads
    char* w = static_cast<char*>(workspace);
    p.part_o = reinterpret_cast<float*>(w);
    p.part_lse = reinterpret_cast<float*>(w + al256((size_t)plan.splits * B * Hkv * 128 * d * 4));
    grid = (long long)B * Hkv * plan.splits;
  }
  if (grid > 0x7fffffffLL) return fail(ATTN_ERR_INVALID_ARG, "problem too large for one launch");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Persistent two-tile kernel (fwd_persist.cu): one CTA per SM walking the same work list.
  const bool persist = !wide && !pack && g_persistent.load() && g_poly.load() == 0;
  // Grouped decode at d = 128: the one-tile kernel (S of the next key block overlaps the
  // softmax of this one) unless the two-tile kernel is chosen.
  const bool pack_one_tile = pack && d == 128 && g_decode_one_tile.load();
  cudaError_t e;
  if (pack_one_tile) {
    e = launch_fwd_wide(maps, p, d, (int)grid, st);
  } else if (persist) {
    p.o_ptr = o;
    const long long entries = grid;
    const long long pgrid = std::min<long long>(entries, std::max(1, s->sms));
    e = launch_fwd_persistent(maps, p, d, (int)pgrid, (int)entries, st);
  } else {
    e = wide ? launch_fwd_wide(maps, p, d, (int)grid, st) : launch_fwd(maps, p, d, pack ? 0 : g_poly.load(), (int)grid, st);
  }
  if (e != cudaSuccess) return cuda_fail(e, "forward launch");
  if (pack && (e = launch_fwd_merge(p, d, o, st)) != cudaSuccess) return cuda_fail(e, "forward merge launch");
  return post_launch(s, st);
}

int attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int N,
             int d, int causal, float scale, void* stream) {
  return fwd_impl(q, k, v, o, lse, B, Hq, Hkv, N, N, d, causal, scale, nullptr, 0, stream);
}

size_t attn_fwd_kv_workspace_size(int B, int Hq, int Hkv, int Nq, int Nk, int d) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || Nq < 0 || Nk < 0 ||
      (d != 64 && d != 128 && d != 192 && d != 256)) {
    set_last_error("attn_fwd_kv_workspace_size: invalid sizes");
    return (size_t)-1;
  }
  const DevSyms* s = dev_syms(nullptr);
  const int sms = s->err == cudaSuccess ? std::max(1, s->sms) : 1;
  return kv_plan(B, Hq, Hkv, Nq, Nk, d, sms).ws_bytes;
}

int attn_fwd_kv(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int Nq,
                int Nk, int d, int causal, float scale, void* workspace, size_t workspace_bytes, void* stream) {
  return fwd_impl(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, workspace, workspace_bytes, stream);
}

// Packed variable-length sequences.  The unit table's size is bounded from the packed
// length alone: sum_b ceil(nq_b / 128) <= floor(total_q / 128) + B tiles per head.
static long long varlen_cap(int B, int Hq, int Hkv, int total_q, int d) {
  const int g = Hq / Hkv;
  const bool pair = g >= 2 && g % 2 == 0;
  const long long tiles = (long long)total_q / 128 + B;
  if (d > 128) return tiles * Hq;   // one tile per record (the one-tile kernel)
  return pair ? tiles * (Hq / 2) : ((tiles + B + 1) / 2) * Hq;
}
static constexpr size_t kVarlenHeader = 256;   // [0] records, [1] offsets invalid

size_t attn_fwd_varlen_workspace_size(int B, int Hq, int Hkv, int total_q, int d) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || total_q < 0 ||
      (d != 64 && d != 128 && d != 192 && d != 256)) {
    set_last_error("attn_fwd_varlen_workspace_size: invalid sizes");
    return (size_t)-1;
  }
  if (B == 0 || total_q == 0) return 0;
  return kVarlenHeader + (size_t)varlen_cap(B, Hq, Hkv, total_q, d) * sizeof(int4);
}

int attn_set_fwd_persistent(int enable) {
  g_persistent.store(enable ? 1 : 0);
  return ATTN_OK;
}

int attn_set_decode_one_tile(int enable) {
  g_decode_one_tile.store(enable ? 1 : 0);
  return ATTN_OK;
}

int attn_set_fwd_one_tile(int enable) {
  g_one_tile_d128.store(enable ? 1 : 0);
  return ATTN_OK;
}

int attn_set_varlen_order(int longest_first) {
  g_varlen_lpt.store(longest_first ? 1 : 0);
  return ATTN_OK;
}

int attn_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse, const int* cu_seqlens_q,
                    const int* cu_seqlens_k, int B, int Hq, int Hkv, int total_q, int total_k, int d, int causal,
                    float scale, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_shape(B, Hq, Hkv, total_q, d, scale, true);
  if (rc != ATTN_OK) return rc;
  if (total_k < 0) return fail(ATTN_ERR_INVALID_ARG, "total_k=%d must be >= 0", total_k);
  if (total_q > 0x7fffff00 || total_k > 0x7fffff00)
    return fail(ATTN_ERR_INVALID_ARG, "packed lengths must stay below 2^31 - 256 rows");
  if (Hq > 65535) return fail(ATTN_ERR_UNSUPPORTED, "Hq=%d: packed sequences support at most 65535 heads", Hq);
  if (B == 0 || total_q == 0) return ATTN_OK;
  if (total_k == 0) return fail(ATTN_ERR_INVALID_ARG, "total_k=0 with %d queries: the softmax has no keys", total_q);
  if (!q || !k || !v || !o || !lse || !cu_seqlens_q || !cu_seqlens_k)
    return fail(ATTN_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return fail(ATTN_ERR_MISALIGNED, "q, k, v, o and lse must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(cu_seqlens_q) | reinterpret_cast<uintptr_t>(cu_seqlens_k)) & 3u)
    return fail(ATTN_ERR_MISALIGNED, "cu_seqlens_q and cu_seqlens_k must be 4-byte aligned");
  const long long cap = varlen_cap(B, Hq, Hkv, total_q, d);
  const size_t need = kVarlenHeader + (size_t)cap * sizeof(int4);
  if (!workspace || workspace_bytes < need)
    return fail(ATTN_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", workspace_bytes, need);
  if (!aligned16(workspace)) return fail(ATTN_ERR_MISALIGNED, "workspace must be 16-byte aligned");
  if (cap > 0x7fffffffLL) return fail(ATTN_ERR_INVALID_ARG, "problem too large for one launch");
  int dev = 0;
  const DevSyms* s = dev_syms(&dev);
  if (s->err != cudaSuccess) return cuda_fail(s->err, "device setup");

  FwdMaps maps;
  if ((rc = make_map(&maps.q, q, d, total_q, Hq, "q")) != ATTN_OK) return rc;
  if ((rc = make_map(&maps.k, k, d, total_k, Hkv, "k")) != ATTN_OK) return rc;
  if ((rc = make_map(&maps.v, v, d, total_k, Hkv, "v")) != ATTN_OK) return rc;
  if ((rc = make_map(&maps.o, o, d, total_q, Hq, "o")) != ATTN_OK) return rc;

  char* w = static_cast<char*>(workspace);
  FwdParams p{};
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.N = total_q; p.g = Hq / Hkv;
  p.Nk = total_k; p.koff = 0;
  p.causal = causal ? 1 : 0;
  p.pair_heads = (p.g >= 2 && p.g % 2 == 0) ? 1 : 0;
  p.pack = 2;
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  p.vl_count = reinterpret_cast<const int*>(w);
  p.vl_units = reinterpret_cast<const int4*>(w + kVarlenHeader);
  p.o_ptr = o;
  p.q_tile_bytes = (unsigned)((d / 64) * 128 * 128);
  p.c = scale * 1.4426950408889634f;
  p.tau = g_tau.load();
  p.lse = lse;
  p.wait_ns = (unsigned long long)g_wait_ns.load();
  p.status = s->status;
  p.rescale_count = g_count_rescales.load() ? s->rescale : nullptr;
  p.test_skip_first_kv = g_test_skip_kv.load();

  VarlenSched sc{};
  sc.cu_q = cu_seqlens_q;
  sc.cu_k = cu_seqlens_k;
  const bool wide = d > 128;        // one query tile per CTA (the one-tile kernel)
  sc.backward = 0;
  sc.single = wide ? 1 : 0;
  sc.B = B; sc.Hq = Hq; sc.Hkv = Hkv; sc.pair_heads = wide ? 0 : p.pair_heads; sc.causal = p.causal;
  sc.total_q = total_q; sc.total_k = total_k;
  sc.nbins = (int)std::min<long long>((total_k + 127LL) / 128 + 1, 32768LL);   // classes: a sequence's key blocks
  sc.cap = (int)cap;
  sc.lpt = g_varlen_lpt.load();
  sc.header = reinterpret_cast<int*>(w);
  sc.units = reinterpret_cast<int4*>(w + kVarlenHeader);
  sc.status = s->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_varlen_schedule(sc, st);
  if (e != cudaSuccess) return cuda_fail(e, "unit table launch");
  e = wide ? launch_fwd_wide(maps, p, d, (int)cap, st) : launch_fwd(maps, p, d, 0, (int)cap, st);
  if (e != cudaSuccess) return cuda_fail(e, "forward launch");
  return post_launch(s, st);
}

int attn_quantize_fp8(const void* x, void* x8, float* scales, int B, int H, int N, int d, void* stream) {
  if (B < 0 || H <= 0 || N < 0) return fail(ATTN_ERR_INVALID_ARG, "B=%d, H=%d, N=%d: need B, N >= 0 and H >= 1", B, H, N);
  if (d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim d=%d (the FP8 path supports 128)", d);
  if (B == 0 || N == 0) return ATTN_OK;
  if ((long long)B * H * ((N + 127) / 128) > 0x7fffffffLL) return fail(ATTN_ERR_INVALID_ARG, "too many blocks");
  if (!x || !x8 || !scales) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(x) || !aligned16(x8) || (reinterpret_cast<uintptr_t>(scales) & 3u))
    return fail(ATTN_ERR_MISALIGNED, "x and x8 must be 16-byte aligned, scales 4-byte aligned");
  cudaError_t e = launch_quantize_fp8(x, x8, scales, (long long)B * H, N, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "quantiser launch");
  return ATTN_OK;
}

int attn_fwd_fp8(const void* q8, const void* k8, const void* v8, const float* q_scale, const float* k_scale,
                 const float* v_scale, void* o, float* lse, int B, int Hq, int Hkv, int N, int d, int causal,
                 float scale, void* stream) {
  int rc = check_shape(B, Hq, Hkv, N, d == 128 ? 128 : 0, scale);
  if (rc != ATTN_OK) {
    if (d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim d=%d (the FP8 path supports 128)", d);
    return rc;
  }
  if (B == 0 || N == 0) return ATTN_OK;
  if (!q8 || !k8 || !v8 || !q_scale || !k_scale || !v_scale || !o || !lse)
    return fail(ATTN_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(q8) || !aligned16(k8) || !aligned16(v8) || !aligned16(o) || !aligned16(lse))
    return fail(ATTN_ERR_MISALIGNED, "q8, k8, v8, o and lse must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(q_scale) | reinterpret_cast<uintptr_t>(k_scale) |
       reinterpret_cast<uintptr_t>(v_scale)) & 3u)
    return fail(ATTN_ERR_MISALIGNED, "the scale arrays must be 4-byte aligned");
  int dev = 0;
  const DevSyms* s = dev_syms(&dev);
  if (s->err != cudaSuccess) return cuda_fail(s->err, "device setup");
  FwdMaps maps;
  if ((rc = make_map_e4m3(&maps.q, q8, N, (long long)B * Hq, "q8")) != ATTN_OK) return rc;
  if ((rc = make_map_e4m3(&maps.k, k8, N, (long long)B * Hkv, "k8")) != ATTN_OK) return rc;
  if ((rc = make_map_e4m3(&maps.v, v8, N, (long long)B * Hkv, "v8")) != ATTN_OK) return rc;
  if ((rc = make_map(&maps.o, o, 128, N, (long long)B * Hq, "o")) != ATTN_OK) return rc;
  FwdParams p{};
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.N = N; p.g = Hq / Hkv;
  p.Nk = N; p.koff = 0;
  p.causal = causal ? 1 : 0;
  p.pair_heads = (p.g >= 2 && p.g % 2 == 0) ? 1 : 0;
  p.n_qblk = (N + 127) / 128;
  p.n_kvblk = p.n_qblk;
  p.n_rowslots = p.pair_heads ? p.n_qblk : (p.n_qblk + 1) / 2;
  p.units_per_row = p.pair_heads ? B * (Hq / 2) : B * Hq;
  p.c = scale * 1.4426950408889634f;
  p.tau = g_tau.load();
  p.lse = lse;
  p.wait_ns = (unsigned long long)g_wait_ns.load();
  p.status = s->status;
  p.rescale_count = g_count_rescales.load() ? s->rescale : nullptr;
  p.test_skip_first_kv = g_test_skip_kv.load();
  // Two-tile units, the last partial wave split into one-tile CTAs (as attn_fwd).
  const long long units = (long long)p.n_rowslots * p.units_per_row;
  p.split_from = (int)std::min<long long>(units, 0x7fffffffLL);
  if (!p.causal) {
    const long long sms = std::max(1, s->sms);
    const long long rem = units % sms;
    if (units >= sms && rem > 0 && 2 * rem <= sms) p.split_from = (int)(units - rem);
    else if (units < sms && 2 * units <= sms) p.split_from = 0;
  }
  const long long grid = p.split_from + 2 * (units - p.split_from);
  if (grid > 0x7fffffffLL) return fail(ATTN_ERR_INVALID_ARG, "problem too large for one launch");
  p.prefetch_ahead = std::max(1, s->sms);
  const Fp8Scales sc{q_scale, k_scale, v_scale};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_fwd_fp8(maps, p, sc, (int)grid, st);
  if (e != cudaSuccess) return cuda_fail(e, "FP8 forward launch");
  return post_launch(s, st);
}

int attn_exp2_sw(const float* x, float* y, long long n, int variant, void* stream) {
  if (n < 0) return fail(ATTN_ERR_INVALID_ARG, "n must be >= 0");
  if (n > 0 && (!x || !y)) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
  if (variant < 0 || variant > 2) return fail(ATTN_ERR_INVALID_ARG, "variant must be 0, 1 or 2");
  cudaError_t e = launch_exp2_test(x, y, n, variant, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "exp2 launch");
  return ATTN_OK;
}

}  // extern "C"

extern "C" {

size_t attn_bwd_workspace_size(int B, int Hq, int Hkv, int N, int d, int deterministic) {
  if (check_shape(B, Hq, Hkv, N, d, 1.0f, true) != ATTN_OK) return (size_t)-1;
  if (B == 0 || N == 0) return 0;
  if (d > 128) return bwd_wide_workspace_bytes(B, Hq, N, d, deterministic);
  // Enough for either query-tile choice (attn_set_bwd_query_tile), so that a workspace sized
  // once serves both.
  return std::max(bwd_workspace_bytes(B, Hq, Hkv, N, d, deterministic),
                  bwd_wide_workspace_bytes(B, Hq, N, d, deterministic));
}

int attn_set_bwd_query_tile(int rows) {
  if (rows != 64 && rows != 128) return fail(ATTN_ERR_INVALID_ARG, "query tile rows=%d (64 or 128)", rows);
  g_bwd_tile_rows.store(rows);
  return ATTN_OK;
}

int attn_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
             void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N, int d, int causal, float scale,
             int deterministic, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_shape(B, Hq, Hkv, N, d, scale, true);
  if (rc != ATTN_OK) return rc;
  if (B == 0 || N == 0) return ATTN_OK;
  // 64-row query tiles (bwd_wide.cu): always for d = 192, 256; for d <= 128 when chosen.
  const bool wide = d > 128 || g_bwd_tile_rows.load() == 64;
  const size_t need = wide ? bwd_wide_workspace_bytes(B, Hq, N, d, deterministic)
                           : bwd_workspace_bytes(B, Hq, Hkv, N, d, deterministic);
  if (!workspace || workspace_bytes < need)
    return fail(ATTN_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", workspace_bytes, need);
  if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv) return fail(ATTN_ERR_INVALID_ARG, "null tensor pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) || !aligned16(dout) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(workspace))
    return fail(ATTN_ERR_MISALIGNED, "every tensor and the workspace must be 16-byte aligned");
  int dev = 0;
  const DevSyms* s = dev_syms(&dev);
  if (s->err != cudaSuccess) return cuda_fail(s->err, "device setup");
  BwdMaps maps;
  const int qrows = wide ? 64 : 128;   // query tile rows of the kernel
  if ((rc = make_map(&maps.q, q, d, N, (long long)B * Hq, "q", qrows)) != ATTN_OK) return rc;
  if ((rc = make_map(&maps.k, k, d, N, (long long)B * Hkv, "k")) != ATTN_OK) return rc;
  if ((rc = make_map(&maps.v, v, d, N, (long long)B * Hkv, "v")) != ATTN_OK) return rc;
  if ((rc = make_map(&maps.dout, dout, d, N, (long long)B * Hq, "dout", qrows)) != ATTN_OK) return rc;
  if ((rc = make_map(&maps.dk, dk, d, N, (long long)B * Hkv, "dk")) != ATTN_OK) return rc;
  if ((rc = make_map(&maps.dv, dv, d, N, (long long)B * Hkv, "dv")) != ATTN_OK) return rc;
  BwdParams p{};
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.N = N; p.g = Hq / Hkv; p.D = d;
  p.causal = causal ? 1 : 0;
  p.deterministic = deterministic ? 1 : 0;
  p.scale = scale;
  p.c = scale * 1.4426950408889634f;
  p.q = q; p.k = k; p.v = v; p.o = o; p.dout = dout; p.lse = lse;
  p.dq = dq; p.dk = dk; p.dv = dv;
  if (wide) bwd_wide_workspace_carve(workspace, B, Hq, N, d, deterministic, &p);
  else bwd_workspace_carve(workspace, B, Hq, Hkv, N, d, deterministic, &p);
  p.wait_ns = (unsigned long long)g_wait_ns.load();
  p.status = s->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = wide ? launch_bwd_wide(maps, p, st) : launch_bwd(maps, p, st);
  if (e == cudaErrorNotSupported) return fail(ATTN_ERR_UNSUPPORTED, "backward not available for these arguments");
  if (e != cudaSuccess) return cuda_fail(e, "backward launch");
  return post_launch(s, st);
}

}  // extern "C"

extern "C" {

size_t attn_bwd_varlen_workspace_size(int B, int Hq, int Hkv, int total_q, int total_k, int d, int deterministic) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || total_q < 0 || total_k < 0 || (d != 64 && d != 128)) {
    set_last_error("attn_bwd_varlen_workspace_size: invalid sizes");
    return (size_t)-1;
  }
  if (B == 0 || (total_q == 0 && total_k == 0)) return 0;
  return bwd_varlen_layout(B, Hq, Hkv, total_q, total_k, d, deterministic).total;
}

int attn_bwd_varlen(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
                    void* dq, void* dk, void* dv, const int* cu_seqlens_q, const int* cu_seqlens_k, int B, int Hq,
                    int Hkv, int total_q, int total_k, int d, int causal, float scale, int deterministic,
                    void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_shape(B, Hq, Hkv, total_q, d, scale);
  if (rc != ATTN_OK) return rc;
  if (total_k < 0) return fail(ATTN_ERR_INVALID_ARG, "total_k=%d must be >= 0", total_k);
  if (total_q > 0x7fffff00 || total_k > 0x7fffff00)
    return fail(ATTN_ERR_INVALID_ARG, "packed lengths must stay below 2^31 - 256 rows");
  if (B == 0 || (total_q == 0 && total_k == 0)) return ATTN_OK;
  if (total_k == 0) return fail(ATTN_ERR_INVALID_ARG, "total_k=0 with %d queries: the softmax has no keys", total_q);
  const BwdVarlenLayout L = bwd_varlen_layout(B, Hq, Hkv, total_q, total_k, d, deterministic);
  if (!workspace || workspace_bytes < L.total)
    return fail(ATTN_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", workspace_bytes, L.total);
  // With no queries at all the query-side tensors are empty and may be NULL.
  if (total_q == 0) {
    q = o = dout = k;
    dq = const_cast<void*>(k);
    lse = static_cast<const float*>(k);
  }
  if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv || !cu_seqlens_q || !cu_seqlens_k)
    return fail(ATTN_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) || !aligned16(dout) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(workspace))
    return fail(ATTN_ERR_MISALIGNED, "every tensor and the workspace must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(cu_seqlens_q) | reinterpret_cast<uintptr_t>(cu_seqlens_k)) & 3u)
    return fail(ATTN_ERR_MISALIGNED, "cu_seqlens_q and cu_seqlens_k must be 4-byte aligned");
  if (L.cap > 0x7fffffffLL || (long long)Hq * L.sem_stride > 0x7fffffffLL)
    return fail(ATTN_ERR_INVALID_ARG, "problem too large for one launch");
  int dev = 0;
  const DevSyms* s = dev_syms(&dev);
  if (s->err != cudaSuccess) return cuda_fail(s->err, "device setup");
  // Tensor maps over the packed views (with no queries, one-row maps that are never read).
  BwdMaps maps;
  const int tq = std::max(total_q, 1), tk = total_k;
  if ((rc = make_map(&maps.q, q, d, tq, Hq, "q")) != ATTN_OK) return rc;
  if ((rc = make_map(&maps.dout, dout, d, tq, Hq, "dout")) != ATTN_OK) return rc;
  if ((rc = make_map(&maps.k, k, d, tk, Hkv, "k")) != ATTN_OK) return rc;
  if ((rc = make_map(&maps.v, v, d, tk, Hkv, "v")) != ATTN_OK) return rc;
  if ((rc = make_map(&maps.dk, dk, d, tk, Hkv, "dk")) != ATTN_OK) return rc;
  if ((rc = make_map(&maps.dv, dv, d, tk, Hkv, "dv")) != ATTN_OK) return rc;

  char* w = static_cast<char*>(workspace);
  BwdParams p{};
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.N = total_q; p.g = Hq / Hkv; p.D = d;
  p.causal = causal ? 1 : 0;
  p.deterministic = deterministic ? 1 : 0;
  p.scale = scale;
  p.c = scale * 1.4426950408889634f;
  p.q = q; p.k = k; p.v = v; p.o = o; p.dout = dout; p.lse = lse;
  p.dq = dq; p.dk = dk; p.dv = dv;
  p.dq_acc = reinterpret_cast<float*>(w + L.dq_acc);
  p.delta = reinterpret_cast<float*>(w + L.delta);
  p.lse2 = reinterpret_cast<float*>(w + L.lse2);
  p.sem = deterministic ? reinterpret_cast<int*>(w + L.sem) : nullptr;
  p.wait_ns = (unsigned long long)g_wait_ns.load();
  p.status = s->status;
  p.varlen = 1;
  p.total_k = total_k;
  p.sem_stride = L.sem_stride;
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  p.vl_count = reinterpret_cast<const int*>(w + L.table);
  p.vl_units = reinterpret_cast<const int4*>(w + L.table + kVarlenHeader);

  VarlenSched sc{};
  sc.cu_q = cu_seqlens_q;
  sc.cu_k = cu_seqlens_k;
  sc.backward = 1;
  sc.B = B; sc.Hq = Hq; sc.Hkv = Hkv; sc.pair_heads = 0; sc.causal = p.causal;
  sc.total_q = total_q; sc.total_k = total_k;
  sc.nbins = (int)std::min<long long>((total_k + 127LL) / 128 + 1, 32768LL);   // classes: a sequence's key blocks
  sc.cap = (int)L.cap;
  sc.lpt = g_varlen_lpt.load();
  sc.header = reinterpret_cast<int*>(w + L.table);
  sc.units = reinterpret_cast<int4*>(w + L.table + kVarlenHeader);
  sc.status = s->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_varlen_schedule(sc, st);
  if (e != cudaSuccess) return cuda_fail(e, "unit table launch");
  e = launch_bwd(maps, p, st);
  if (e == cudaErrorNotSupported) return fail(ATTN_ERR_UNSUPPORTED, "backward not available for these arguments");
  if (e != cudaSuccess) return cuda_fail(e, "backward launch");
  return post_launch(s, st);
}

}  // extern "C"

extern "C" {

// Whether rows of d elements at these strides lie apart: in ascending order, every stride in use reaches
// past all that the smaller ones span.
static bool rows_apart(const int (&extent)[3], const long long (&stride)[3], int d) {
  __int128 step[3];
  int order[3] = {0, 1, 2};
  for (int a = 0; a < 3; ++a) step[a] = stride[a] < 0 ? -(__int128)stride[a] : (__int128)stride[a];
  std::sort(order, order + 3, [&](int a, int b) { return step[a] < step[b]; });
  __int128 span = d;
  for (int a : order) {
    if (extent[a] <= 1) continue;
    if (step[a] < span) return false;
    span += (extent[a] - 1) * step[a];
  }
  return true;
}

// strides: {q, k, q_out, k_out} x {batch, head, token} in elements, or null for contiguous
// [B, H, N, d] tensors.
// Checks the arguments and fills in *p and the elements per access; *nothing: an empty call.
static int rope_params(const void* q, const void* k, void* q_out, void* k_out, const double* inv_freq,
                       const int* positions, int B, int Hq, int Hk, int N, int d, int rot, float mscale,
                       const long long* strides, int backward, RopeParams* out, int* vec, bool* nothing) {
  *nothing = false;
  if (B < 0 || N < 0) return fail(ATTN_ERR_INVALID_ARG, "B=%d and N=%d must be >= 0", B, N);
  if (Hq <= 0 || Hk < 0) return fail(ATTN_ERR_INVALID_ARG, "Hq=%d must be >= 1 and Hk=%d >= 0", Hq, Hk);
  if (d != 64 && d != 128 && d != 192 && d != 256)
    return fail(ATTN_ERR_UNSUPPORTED, "head dim d=%d (supported: 64, 128, 192, 256)", d);
  if (rot < 2 || rot > d || (rot & 1))
    return fail(ATTN_ERR_INVALID_ARG, "rot=%d must be even and between 2 and d=%d", rot, d);
  if (!std::isfinite(mscale)) return fail(ATTN_ERR_INVALID_ARG, "mscale must be finite");
  if (N > 0x7fff0000) return fail(ATTN_ERR_INVALID_ARG, "N must stay below 2^31 - 65536");
  if ((long long)Hq + Hk > 65535) return fail(ATTN_ERR_INVALID_ARG, "Hq + Hk too large");
  if (B == 0 || N == 0) {
    *nothing = true;
    return ATTN_OK;
  }
  if (!q || !q_out || !inv_freq || (Hk > 0 && (!k || !k_out))) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
  RopeParams& p = *out;
  p = RopeParams{};
  p.q.in = q; p.q.out = q_out; p.k.in = k; p.k.out = k_out;
  const long long cq[3] = {(long long)Hq * N * d, (long long)N * d, d}, ck[3] = {(long long)Hk * N * d, (long long)N * d, d};
  const long long* sq = strides ? strides : cq;
  const long long* sk = strides ? strides + 3 : ck;
  const long long* oq = strides ? strides + 6 : cq;
  const long long* ok = strides ? strides + 9 : ck;
  p.q.in_b = sq[0]; p.q.in_h = sq[1]; p.q.in_n = sq[2]; p.q.out_b = oq[0]; p.q.out_h = oq[1]; p.q.out_n = oq[2];
  p.k.in_b = sk[0]; p.k.in_h = sk[1]; p.k.in_n = sk[2]; p.k.out_b = ok[0]; p.k.out_h = ok[1]; p.k.out_n = ok[2];
  uintptr_t bits = 0;
  const int ext[2][3] = {{B, Hq, N}, {B, Hk, N}};
  for (int i = 0; i < (Hk > 0 ? 2 : 1); ++i) {
    const RopeTensor& t = i ? p.k : p.q;
    const long long in[3] = {t.in_b, t.in_h, t.in_n}, out[3] = {t.out_b, t.out_h, t.out_n};
    bits |= reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out);
    for (int a = 0; a < 3; ++a) {
      if (ext[i][a] <= 1) continue;                    // the stride is not used
      bits |= (uintptr_t)(in[a] * 2) | (uintptr_t)(out[a] * 2);
      if (t.in == t.out && in[a] != out[a])
        return fail(ATTN_ERR_INVALID_ARG, "in place needs equal strides of input and output");
    }
    if (!rows_apart(ext[i], out, d))
      return fail(ATTN_ERR_INVALID_ARG, "output rows overlap (strides %lld, %lld, %lld)", out[0], out[1], out[2]);
  }
  if (bits & 1) return fail(ATTN_ERR_MISALIGNED, "bf16 tensors must be 2-byte aligned");
  if ((reinterpret_cast<uintptr_t>(inv_freq) & 7u) || (reinterpret_cast<uintptr_t>(positions) & 3u))
    return fail(ATTN_ERR_MISALIGNED, "inv_freq must be 8-byte aligned, positions 4-byte aligned");
  *vec = (bits & 15) == 0 && rot % 16 == 0 ? 8 : ((bits & 7) == 0 && rot % 8 == 0 ? 4 : 1);
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.B = B; p.N = N; p.Hq = Hq; p.Hk = Hk; p.d = d; p.rot = rot;
  p.mscale = mscale;
  p.sign = backward ? -1.f : 1.f;
  return ATTN_OK;
}

static int rope_impl(const void* q, const void* k, void* q_out, void* k_out, const double* inv_freq,
                     const int* positions, int B, int Hq, int Hk, int N, int d, int rot, int interleaved, float mscale,
                     const long long* strides, int backward, void* stream) {
  RopeParams p;
  int vec;
  bool nothing;
  const int rc = rope_params(q, k, q_out, k_out, inv_freq, positions, B, Hq, Hk, N, d, rot, mscale, strides, backward, &p,
                             &vec, &nothing);
  if (rc != ATTN_OK || nothing) return rc;
  const DevSyms* s = dev_syms(nullptr);
  if (s->err != cudaSuccess) return cuda_fail(s->err, "device setup");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_rope(p, vec, interleaved ? 1 : 0, std::max(1, s->sms), st);
  if (e != cudaSuccess) return cuda_fail(e, "rotary launch");
  return post_launch(s, st);
}

int attn_rope(const void* q, const void* k, void* q_out, void* k_out, const double* inv_freq, const int* positions,
              int B, int Hq, int Hk, int N, int d, int rot, int interleaved, float mscale, const long long* strides,
              void* stream) {
  return rope_impl(q, k, q_out, k_out, inv_freq, positions, B, Hq, Hk, N, d, rot, interleaved, mscale, strides, 0,
                   stream);
}

int attn_rope_bwd(const void* dq, const void* dk, void* dq_out, void* dk_out, const double* inv_freq,
                  const int* positions, int B, int Hq, int Hk, int N, int d, int rot, int interleaved, float mscale,
                  const long long* strides, void* stream) {
  return rope_impl(dq, dk, dq_out, dk_out, inv_freq, positions, B, Hq, Hk, N, d, rot, interleaved, mscale, strides, 1,
                   stream);
}

// Sizes common to the paged cache's calls.
static int check_cache(int B, int Hkv, int total, int d, int num_pages, int page_size, int max_pages) {
  if (B < 0 || total < 0) return fail(ATTN_ERR_INVALID_ARG, "B=%d and the packed length %d must be >= 0", B, total);
  if (B == 0 && total > 0) return fail(ATTN_ERR_INVALID_ARG, "%d packed rows but no sequence", total);
  if (Hkv <= 0 || Hkv > 65535) return fail(ATTN_ERR_INVALID_ARG, "Hkv=%d must be between 1 and 65535", Hkv);
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim d=%d (the 8-bit cache supports 64, 128)", d);
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return fail(ATTN_ERR_UNSUPPORTED, "page size %d (supported: 16, 32, 64, 128)", page_size);
  if (num_pages < 0 || max_pages < 0) return fail(ATTN_ERR_INVALID_ARG, "page counts must be >= 0");
  if ((long long)max_pages * page_size > 0x7fff0000LL)
    return fail(ATTN_ERR_INVALID_ARG, "max_pages * page_size must stay below 2^31 - 65536");
  if (total > 0x7fff0000) return fail(ATTN_ERR_INVALID_ARG, "packed length must stay below 2^31 - 65536");
  if ((long long)num_pages * Hkv > 0x7fffffffLL) return fail(ATTN_ERR_INVALID_ARG, "num_pages * Hkv too large");
  return ATTN_OK;
}
static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Checks of an append's rows and cache, and its parameters.
static int append_params(const void* k, const void* v, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                         const int* page_table, const int* cu_seqlens, const int* kv_lens, int B, int Hkv, int total, int d,
                         int num_pages, int page_size, int max_pages, const long long (&st4)[4], AppendParams* out) {
  if (num_pages == 0 || max_pages == 0) return fail(ATTN_ERR_INVALID_ARG, "%d rows to append, but no pages", total);
  if (!k || !v || !k_cache || !v_cache || !k_scale || !v_scale || !page_table || !cu_seqlens || !kv_lens)
    return fail(ATTN_ERR_INVALID_ARG, "null pointer");
  uintptr_t bits = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v);
  for (int i = 0; i < 4; ++i)
    if ((i & 1 ? total : Hkv) > 1) bits |= (uintptr_t)(st4[i] * 2);
  if ((bits & 15) || !aligned16(k_cache) || !aligned16(v_cache))
    return fail(ATTN_ERR_MISALIGNED, "k, v (their strides too) and the cache must be 16-byte aligned");
  if (!aligned4(k_scale) || !aligned4(v_scale) || !aligned4(page_table) || !aligned4(cu_seqlens) || !aligned4(kv_lens))
    return fail(ATTN_ERR_MISALIGNED, "scales, page table, offsets and lengths must be 4-byte aligned");
  AppendParams& p = *out;
  p = AppendParams{};
  p.k = k; p.v = v;
  p.k_h = st4[0]; p.k_t = st4[1]; p.v_h = st4[2]; p.v_t = st4[3];
  p.k_cache = k_cache; p.v_cache = v_cache; p.k_scale = k_scale; p.v_scale = v_scale;
  p.table = page_table; p.cu = cu_seqlens; p.kv_lens = kv_lens;
  p.B = B; p.Hkv = Hkv; p.total = total; p.num_pages = num_pages; p.page = page_size; p.max_pages = max_pages;
  p.max_len = max_pages * page_size;
  return ATTN_OK;
}

// strides: {k head, k token, v head, v token} in elements, or null for contiguous [Hkv, total, d].
int attn_kv_append_fp8(const void* k, const void* v, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                       const int* page_table, const int* cu_seqlens, const int* kv_lens, int B, int Hkv, int total,
                       int d, int num_pages, int page_size, int max_pages, const long long* strides, void* stream) {
  int rc = check_cache(B, Hkv, total, d, num_pages, page_size, max_pages);
  if (rc != ATTN_OK) return rc;
  if (B == 0 || total == 0) return ATTN_OK;
  const long long td = (long long)total * d;
  const long long st4[4] = {strides ? strides[0] : td, strides ? strides[1] : d, strides ? strides[2] : td,
                            strides ? strides[3] : d};
  AppendParams p;
  rc = append_params(k, v, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens, kv_lens, B, Hkv, total, d, num_pages,
                     page_size, max_pages, st4, &p);
  if (rc != ATTN_OK) return rc;
  const DevSyms* s = dev_syms(nullptr);
  if (s->err != cudaSuccess) return cuda_fail(s->err, "device setup");
  p.status = s->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_kv_append(p, d, std::max(1, s->sms), st);
  if (e != cudaSuccess) return cuda_fail(e, "cache append launch");
  return post_launch(s, st);
}

// strides: {q head, q token, k head, k token, v head, v token, q_out head, q_out token} in elements, or null.
int attn_rope_kv_append_fp8(const void* q, void* q_out, const void* k, const void* v, const double* inv_freq,
                            const int* positions, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                            void* k_bounds, const int* page_table, const int* cu_seqlens, const int* kv_lens, int B, int Hq,
                            int Hkv, int total, int d, int rot, int interleaved, float mscale, int num_pages, int page_size,
                            int max_pages, const long long* strides, void* stream) {
  int rc = check_cache(B, Hkv, total, d, num_pages, page_size, max_pages);
  if (rc != ATTN_OK) return rc;
  if (rot < 0 || rot > d || (rot & 1)) return fail(ATTN_ERR_INVALID_ARG, "rot=%d must be even and between 0 and d=%d", rot, d);
  if (!std::isfinite(mscale)) return fail(ATTN_ERR_INVALID_ARG, "mscale must be finite");
  if (Hq < 0) return fail(ATTN_ERR_INVALID_ARG, "Hq=%d must be >= 0", Hq);
  if (Hq > 0 && rot == 0) return fail(ATTN_ERR_INVALID_ARG, "rot = 0 leaves the queries as they are: pass none (Hq = 0)");
  if (B == 0 || total == 0) return ATTN_OK;
  const long long td = (long long)total * d;
  const long long contiguous[8] = {td, d, td, d, td, d, td, d};
  const long long* st8 = strides ? strides : contiguous;
  const long long st4[4] = {st8[2], st8[3], st8[4], st8[5]};
  RopeAppendParams p{};
  rc = append_params(k, v, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens, kv_lens, B, Hkv, total, d, num_pages,
                     page_size, max_pages, st4, &p.a);
  if (rc != ATTN_OK) return rc;
  if (rot > 0 && !inv_freq) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
  if ((reinterpret_cast<uintptr_t>(inv_freq) & 7u) || !aligned4(positions))
    return fail(ATTN_ERR_MISALIGNED, "inv_freq must be 8-byte aligned, positions 4-byte aligned");
  if (!aligned16(k_bounds)) return fail(ATTN_ERR_MISALIGNED, "k_bounds must be 16-byte aligned");
  RopeParams r{};
  int vec = 1;
  if (Hq > 0) {
    const long long st12[12] = {0, st8[0], st8[1], 0, 0, 0, 0, st8[6], st8[7], 0, 0, 0};
    bool nothing;
    rc = rope_params(q, nullptr, q_out, nullptr, inv_freq, positions, 1, Hq, 0, total, d, rot, mscale, st12, 0, &r, &vec,
                     &nothing);
    if (rc != ATTN_OK) return rc;
    r.cu = cu_seqlens;
    r.kv_lens = kv_lens;
    r.seqs = B;
  }
  const DevSyms* s = dev_syms(nullptr);
  if (s->err != cudaSuccess) return cuda_fail(s->err, "device setup");
  p.a.status = s->status;
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.rot = rot;
  p.interleaved = interleaved ? 1 : 0;
  p.mscale = mscale;
  p.bounds = static_cast<uint8_t*>(k_bounds);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  bool queries = Hq > 0 && rot % 8 == 0 && aligned16(q) && aligned16(q_out);
  for (int i : {0, 1, 6, 7}) queries = queries && ((i & 1 ? total : Hq) <= 1 || st8[i] % 8 == 0);
  p.q = q;
  p.q_out = q_out;
  p.q_h = st8[0]; p.q_t = st8[1]; p.o_h = st8[6]; p.o_t = st8[7];
  p.Hq = Hq;
  cudaError_t e = launch_rope_append(p, d, std::max(1, s->sms), &queries, st);
  if (e == cudaSuccess && Hq > 0 && !queries) e = launch_rope(r, vec, p.interleaved, std::max(1, s->sms), st);
  if (e != cudaSuccess) return cuda_fail(e, "rotating cache append launch");
  return post_launch(s, st);
}

static size_t cache_workspace_bytes(int Hq, int Hkv, int max_q, int d, int sms) {
  const long long rows = (long long)max_q * (Hq / Hkv);
  return rows <= kCacheDecodeRows ? cache_decode_workspace_bytes((int)rows, d, sms) : cache_tile_workspace_bytes(d, sms);
}

size_t attn_fwd_kv_fp8_workspace_size(int B, int Hq, int Hkv, int total_q, int max_q, int d) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || total_q < 0 || max_q < 0 || (d != 64 && d != 128)) {
    set_last_error("attn_fwd_kv_fp8_workspace_size: invalid sizes");
    return (size_t)-1;
  }
  if (B == 0 || total_q == 0) return 0;
  const DevSyms* s = dev_syms(nullptr);
  const int sms = s->err == cudaSuccess ? std::max(1, s->sms) : 1;
  return cache_workspace_bytes(Hq, Hkv, max_q, d, sms);
}

// The checks and parameters that the calls of attention over the cache share.
struct CacheCall {
  const void *q, *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int *page_table, *cu_seqlens_q, *kv_lens;
  void* o;
  float* lse;
  int B, Hq, Hkv, total_q, d, num_pages, page_size, max_pages, causal;
  float scale;
};
static int check_cache_call(const CacheCall& c) {
  int rc = check_cache(c.B, c.Hkv, c.total_q, c.d, c.num_pages, c.page_size, c.max_pages);
  if (rc != ATTN_OK) return rc;
  if ((rc = check_shape(c.B, c.Hq, c.Hkv, c.total_q, c.d, c.scale)) != ATTN_OK) return rc;
  if (c.Hq > 65535) return fail(ATTN_ERR_UNSUPPORTED, "Hq=%d: packed sequences support at most 65535 heads", c.Hq);
  if (c.Hq / c.Hkv > 256) return fail(ATTN_ERR_UNSUPPORTED, "Hq / Hkv = %d (supported: up to 256)", c.Hq / c.Hkv);
  if (c.B == 0 || c.total_q == 0) return ATTN_OK;
  if (c.num_pages == 0) return fail(ATTN_ERR_INVALID_ARG, "%d queries, but no pages", c.total_q);
  return ATTN_OK;
}
static int check_max_q(const char* name, int max_q, int total_q) {
  if (max_q < 1 || max_q > total_q)
    return fail(ATTN_ERR_INVALID_ARG,
                "%s=%d must be between 1 and the %d packed queries (of a constant bound and these pass the smaller)",
                name, max_q, total_q);
  return ATTN_OK;
}
static int check_cache_pointers(const CacheCall& c) {
  // (A table without columns, whose lengths are all 0, is never read.)
  if (!c.q || !c.k_cache || !c.v_cache || !c.k_scale || !c.v_scale || (!c.page_table && c.max_pages > 0) ||
      !c.cu_seqlens_q || !c.kv_lens || !c.o || !c.lse)
    return fail(ATTN_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(c.q) || !aligned16(c.o) || !aligned16(c.k_cache) || !aligned16(c.v_cache))
    return fail(ATTN_ERR_MISALIGNED, "q, o and the cache must be 16-byte aligned");
  if (!aligned4(c.k_scale) || !aligned4(c.v_scale) || !aligned4(c.page_table) || !aligned4(c.cu_seqlens_q) ||
      !aligned4(c.kv_lens) || !aligned4(c.lse))
    return fail(ATTN_ERR_MISALIGNED, "scales, page table, offsets, lengths and lse must be 4-byte aligned");
  return ATTN_OK;
}
static int check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (!workspace || bytes < need) return fail(ATTN_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", bytes, need);
  if (!aligned16(workspace)) return fail(ATTN_ERR_MISALIGNED, "workspace must be 16-byte aligned");
  return ATTN_OK;
}
static CacheParams cache_params(const CacheCall& c, int max_q, void* workspace, const DevSyms* s) {
  CacheParams p{};
  p.q = c.q;
  p.k_cache = static_cast<const uint8_t*>(c.k_cache);
  p.v_cache = static_cast<const uint8_t*>(c.v_cache);
  p.k_scale = c.k_scale; p.v_scale = c.v_scale;
  p.table = c.page_table; p.cu_q = c.cu_seqlens_q; p.kv_lens = c.kv_lens;
  p.o = c.o; p.lse = c.lse;
  p.B = c.B; p.Hq = c.Hq; p.Hkv = c.Hkv; p.g = c.Hq / c.Hkv; p.total_q = c.total_q; p.max_q = max_q;
  p.num_pages = c.num_pages; p.page = c.page_size; p.max_pages = c.max_pages; p.max_len = c.max_pages * c.page_size;
  p.causal = c.causal ? 1 : 0;
  p.c = c.scale * 1.4426950408889634f;
  p.ws = workspace;
  p.wait_ns = (unsigned long long)g_wait_ns.load();
  p.status = s->status;
  p.test_skip_first_kv = g_test_skip_kv.load();
  return p;
}
// few: the kernels for few rows (pieces of 32 keys), else the tiles (blocks of 128).
static int cache_maps(const CacheCall& c, bool few, CacheMaps* maps) {
  const int box = std::min(c.page_size, few ? 32 : 128), d = c.d;      // keys per copy
  const long long slabs = (long long)c.num_pages * c.Hkv;
  const int kline = few ? 128 : d;
  const int rc = make_map_cache(&maps->k, c.k_cache, kline, c.page_size * d / kline, slabs, box * d / kline, "k_cache");
  if (rc != ATTN_OK) return rc;
  return make_map_cache(&maps->v, c.v_cache, 128, c.page_size * d / 128, slabs, box * d / 128, "v_cache");
}
static bool few_rows(const CacheParams& p) { return (long long)p.max_q * p.g <= kCacheDecodeRows; }
static int launch_cache(const CacheMaps& maps, const CacheParams& p, int d, int sms, cudaStream_t st) {
  const cudaError_t e = few_rows(p) ? launch_fwd_cache_decode(maps, p, d, sms, st) : launch_fwd_cache_tile(maps, p, d, sms, st);
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "cached attention launch");
}

int attn_fwd_kv_fp8(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                    const float* v_scale, const int* page_table, const int* cu_seqlens_q, const int* kv_lens, void* o,
                    float* lse, int B, int Hq, int Hkv, int total_q, int max_q, int d, int num_pages, int page_size,
                    int max_pages, int causal, float scale, void* workspace, size_t workspace_bytes, void* stream) {
  const CacheCall c{q, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens_q, kv_lens, o, lse,
                    B, Hq, Hkv, total_q, d, num_pages, page_size, max_pages, causal, scale};
  int rc = check_cache_call(c);
  if (rc != ATTN_OK || B == 0 || total_q == 0) return rc;
  if ((rc = check_max_q("max_q", max_q, total_q)) != ATTN_OK) return rc;
  if ((rc = check_cache_pointers(c)) != ATTN_OK) return rc;
  const DevSyms* s = dev_syms(nullptr);
  const int sms = s->err == cudaSuccess ? std::max(1, s->sms) : 1;
  if ((rc = check_workspace(workspace, workspace_bytes, cache_workspace_bytes(Hq, Hkv, max_q, d, sms))) != ATTN_OK) return rc;
  if (s->err != cudaSuccess) return cuda_fail(s->err, "device setup");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const CacheParams p = cache_params(c, max_q, workspace, s);
  CacheMaps maps;
  if ((rc = cache_maps(c, few_rows(p), &maps)) != ATTN_OK) return rc;
  if ((rc = launch_cache(maps, p, d, sms, st)) != ATTN_OK) return rc;
  return post_launch(s, st);
}

// Entries of a list: kernels step up to 1024 past its end, in 32 bits.
constexpr int kMaxListed = 0x7fff0000;
// A block chooses a list (and the workspace's size stays within 64 bits).
static bool few_lists(int Hkv, int total_q) { return (long long)Hkv * total_q <= 0x7fffffffLL; }

size_t attn_select_pages_fp8_workspace_size(int Hkv, int total_q, int max_pages) {
  if (Hkv <= 0 || total_q < 0 || max_pages < 0 || !few_lists(Hkv, total_q) || max_pages > kMaxListed / 16) {
    set_last_error("attn_select_pages_fp8_workspace_size: invalid sizes");
    return (size_t)-1;
  }
  return total_q == 0 || max_pages == 0 ? 0 : select_ws(Hkv, total_q, max_pages).total;
}

int attn_select_pages_fp8(const void* q, const void* k_bounds, const float* k_scale, const int* page_table,
                          const int* cu_seqlens_q, const int* kv_lens, int* pages, int B, int Hq, int Hkv, int total_q,
                          int max_q, int d, int num_pages, int page_size, int max_pages, int count, int first, int last,
                          int causal, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_cache(B, Hkv, total_q, d, num_pages, page_size, max_pages);
  if (rc != ATTN_OK) return rc;
  if ((rc = check_shape(B, Hq, Hkv, total_q, d, 1.f)) != ATTN_OK) return rc;
  if (Hq > 65535) return fail(ATTN_ERR_UNSUPPORTED, "Hq=%d: packed sequences support at most 65535 heads", Hq);
  if (Hq / Hkv > 256) return fail(ATTN_ERR_UNSUPPORTED, "Hq / Hkv = %d (supported: up to 256)", Hq / Hkv);
  if (count < 1 || first < 0 || last < 0 || first > count || last > count - first)
    return fail(ATTN_ERR_INVALID_ARG, "count=%d must be >= 1, first=%d and last=%d >= 0 and together within it", count, first,
                last);
  if (!few_lists(Hkv, total_q))
    return fail(ATTN_ERR_UNSUPPORTED, "Hkv * total_q = %lld lists (supported: below 2^31)", (long long)Hkv * total_q);
  if (count > kMaxListed) return fail(ATTN_ERR_INVALID_ARG, "count=%d must be at most 2^31 - 65536", count);
  if (B == 0 || total_q == 0) return ATTN_OK;
  if (num_pages == 0) return fail(ATTN_ERR_INVALID_ARG, "%d queries, but no pages", total_q);
  if ((rc = check_max_q("max_q", max_q, total_q)) != ATTN_OK) return rc;
  if (!q || !k_bounds || !k_scale || (!page_table && max_pages > 0) || !cu_seqlens_q || !kv_lens || !pages)
    return fail(ATTN_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(q) || !aligned16(k_bounds)) return fail(ATTN_ERR_MISALIGNED, "q and k_bounds must be 16-byte aligned");
  if (!aligned4(k_scale) || !aligned4(page_table) || !aligned4(cu_seqlens_q) || !aligned4(kv_lens) || !aligned4(pages))
    return fail(ATTN_ERR_MISALIGNED, "scales, page table, offsets, lengths and pages must be 4-byte aligned");
  const SelectWs w = select_ws(Hkv, total_q, max_pages);
  if (max_pages > 0 && (rc = check_workspace(workspace, workspace_bytes, w.total)) != ATTN_OK) return rc;
  const DevSyms* s = dev_syms(nullptr);
  if (s->err != cudaSuccess) return cuda_fail(s->err, "device setup");
  char* ws = static_cast<char*>(workspace);
  SelectParams p{};
  p.q = q;
  p.bounds = static_cast<const uint8_t*>(k_bounds);
  p.k_scale = k_scale;
  p.table = page_table; p.cu_q = cu_seqlens_q; p.kv_lens = kv_lens;
  p.out = pages;
  p.B = B; p.Hkv = Hkv; p.g = Hq / Hkv; p.total_q = total_q; p.max_q = max_q;
  p.num_pages = num_pages; p.page = page_size; p.max_pages = max_pages; p.max_len = max_pages * page_size;
  p.count = count; p.first = first; p.last = last;
  p.causal = causal ? 1 : 0;
  p.scores = reinterpret_cast<float*>(ws);
  p.exact = reinterpret_cast<unsigned long long*>(ws + w.exact);
  p.near = reinterpret_cast<int*>(ws + w.near);
  p.errors = reinterpret_cast<float*>(ws + w.errors);
  p.status = s->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_select_pages(p, d, std::max(1, s->sms), st);
  if (e != cudaSuccess) return cuda_fail(e, "page selection launch");
  return post_launch(s, st);
}

// Query heads that one unit of the listed pages' kernel holds: a group's, or its largest share of at most 16.
static int list_group(int g) {
  int share = std::min(g, kCacheDecodeRows);
  while (g % share != 0) --share;
  return share;
}

size_t attn_fwd_kv_fp8_pages_workspace_size(int Hq, int Hkv, int total_q, int d) {
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || total_q < 0 || (d != 64 && d != 128)) {
    set_last_error("attn_fwd_kv_fp8_pages_workspace_size: invalid sizes");
    return (size_t)-1;
  }
  if (total_q == 0) return 0;
  const DevSyms* s = dev_syms(nullptr);
  return cache_decode_workspace_bytes(list_group(Hq / Hkv), d, s->err == cudaSuccess ? std::max(1, s->sms) : 1);
}

int attn_fwd_kv_fp8_pages(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                          const float* v_scale, const int* page_table, const int* cu_seqlens_q, const int* kv_lens,
                          const int* pages, void* o, float* lse, int B, int Hq, int Hkv, int total_q, int count, int d,
                          int num_pages, int page_size, int max_pages, int causal, float scale, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const CacheCall c{q, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens_q, kv_lens, o, lse,
                    B, Hq, Hkv, total_q, d, num_pages, page_size, max_pages, causal, scale};
  int rc = check_cache_call(c);
  if (rc != ATTN_OK) return rc;
  if (count < 0 || count > kMaxListed)
    return fail(ATTN_ERR_INVALID_ARG, "count=%d must be between 0 and 2^31 - 65536", count);
  if (B == 0 || total_q == 0) return ATTN_OK;
  if ((rc = check_cache_pointers(c)) != ATTN_OK) return rc;
  if (count > 0 && !pages) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
  if (!aligned4(pages)) return fail(ATTN_ERR_MISALIGNED, "pages must be 4-byte aligned");
  const DevSyms* s = dev_syms(nullptr);
  const int sms = s->err == cudaSuccess ? std::max(1, s->sms) : 1, share = list_group(Hq / Hkv);
  if ((rc = check_workspace(workspace, workspace_bytes, cache_decode_workspace_bytes(share, d, sms))) != ATTN_OK) return rc;
  if (s->err != cudaSuccess) return cuda_fail(s->err, "device setup");
  CacheParams p = cache_params(c, total_q, workspace, s);
  p.list = pages;
  p.list_count = count;
  p.rep = Hq / Hkv / share;
  p.Hkv = Hkv * p.rep;
  p.g = share;
  CacheMaps maps;
  if ((rc = cache_maps(c, true, &maps)) != ATTN_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_fwd_cache_pages(maps, p, d, sms, st);
  if (e != cudaSuccess) return cuda_fail(e, "listed pages attention launch");
  return post_launch(s, st);
}

// The parts' workspace for partial results (used one after the other, or by one launch), then the parts' results and
// whether their offsets were valid.
struct PrefixWs {
  size_t lse[2], o[2], bad, total;
};
static PrefixWs prefix_ws(int Hq, int Hkv, int total_q, int max_prefix_q, int max_q, int d, int sms) {
  PrefixWs w;
  const auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  size_t at = up(std::max(cache_workspace_bytes(Hq, Hkv, max_prefix_q, d, sms), cache_workspace_bytes(Hq, Hkv, max_q, d, sms)));
  for (int i = 0; i < 2; ++i) {
    w.lse[i] = at;
    w.o[i] = w.lse[i] + up((size_t)Hq * total_q * 4);
    at = w.o[i] + up((size_t)Hq * total_q * d * 4);
  }
  w.bad = at;
  w.total = w.bad + 256;
  return w;
}

size_t attn_fwd_kv_fp8_prefix_workspace_size(int Hq, int Hkv, int total_q, int max_prefix_q, int max_q, int d) {
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || total_q < 0 || max_prefix_q < 0 || max_q < 0 || (d != 64 && d != 128)) {
    set_last_error("attn_fwd_kv_fp8_prefix_workspace_size: invalid sizes");
    return (size_t)-1;
  }
  if (total_q == 0) return 0;
  const DevSyms* s = dev_syms(nullptr);
  return prefix_ws(Hq, Hkv, total_q, max_prefix_q, max_q, d, s->err == cudaSuccess ? std::max(1, s->sms) : 1).total;
}

int attn_fwd_kv_fp8_prefix(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                           const float* v_scale, const int* prefix_table, const int* cu_prefix_q, const int* prefix_lens,
                           const int* page_table, const int* cu_seqlens_q, const int* kv_lens, void* o, float* lse, int G,
                           int B, int Hq, int Hkv, int total_q, int max_prefix_q, int max_q, int d, int num_pages,
                           int page_size, int max_prefix_pages, int max_pages, int causal, float scale, void* workspace,
                           size_t workspace_bytes, void* stream) {
  const CacheCall shared{q, k_cache, v_cache, k_scale, v_scale, prefix_table, cu_prefix_q, prefix_lens, o, lse,
                         G, Hq, Hkv, total_q, d, num_pages, page_size, max_prefix_pages, 0, scale};
  const CacheCall mine{q, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens_q, kv_lens, o, lse,
                       B, Hq, Hkv, total_q, d, num_pages, page_size, max_pages, causal, scale};
  int rc = check_cache_call(shared);
  if (rc != ATTN_OK || (rc = check_cache_call(mine)) != ATTN_OK || total_q == 0) return rc;
  if ((rc = check_max_q("max_prefix_q", max_prefix_q, total_q)) != ATTN_OK) return rc;
  if ((rc = check_max_q("max_q", max_q, total_q)) != ATTN_OK) return rc;
  if ((rc = check_cache_pointers(shared)) != ATTN_OK || (rc = check_cache_pointers(mine)) != ATTN_OK) return rc;
  const DevSyms* s = dev_syms(nullptr);
  const int sms = s->err == cudaSuccess ? std::max(1, s->sms) : 1;
  const PrefixWs w = prefix_ws(Hq, Hkv, total_q, max_prefix_q, max_q, d, sms);
  if ((rc = check_workspace(workspace, workspace_bytes, w.total)) != ATTN_OK) return rc;
  if (s->err != cudaSuccess) return cuda_fail(s->err, "device setup");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CacheParams p[2] = {cache_params(shared, max_prefix_q, workspace, s), cache_params(mine, max_q, workspace, s)};
  char* ws = static_cast<char*>(workspace);
  for (int i = 0; i < 2; ++i) {
    for (int k = 0; k < 2; ++k) {
      p[i].side_lse[k] = reinterpret_cast<float*>(ws + w.lse[k]);
      p[i].side_o[k] = reinterpret_cast<float*>(ws + w.o[k]);
    }
    p[i].side_bad = reinterpret_cast<int*>(ws + w.bad);
    p[i].side = i == 0 ? SIDE_OUT : SIDE_IN;
  }
  CacheMaps maps[2];
  if ((rc = cache_maps(mine, few_rows(p[0]), &maps[0])) != ATTN_OK) return rc;
  // One kernel for both parts, then one that joins them, where the same one suits both (prefixes of 5000 and 16001 keys
  // before 24 pieces of up to 60 queries, 16 heads on 2, d = 64: 67 us against 85 one after the other); and where the
  // sequences' own part has few rows and no more units than there are SMs, so that two main launches' starts count.  One
  // token of each sequence behind 8192 keys, 4 heads to a K/V head, in a graph, by tiles against two launches:
  //   own keys                16        260       2000      16000
  //   10 x 4 K/V heads        31, 41    30, 36    33, 38     65, 69
  //    8 x 8                  39, 41    33, 36    37, 39     90, 85
  //   16 x 8                  34, 42    38, 38    47, 48    151, 128
  //   64 x 2                  38, 47    41, 42    54, 51    218, 133
  // (38 x 8, beyond the rule: 59 against 49.)  So long own keys behind a short prefix lose by it where units are many; the
  // lengths that decide it are on the device.
  const bool tiles = !few_rows(p[0]) && (!few_rows(p[1]) || (long long)B * Hkv <= sms);
  if (tiles || (few_rows(p[0]) && few_rows(p[1]))) {
    p[0].side = SIDE_BOTH;
    p[0].two = {page_table, cu_seqlens_q, kv_lens, B, max_q, max_pages, max_pages * page_size, causal ? 1 : 0};
    if ((rc = launch_cache(maps[0], p[0], d, sms, st)) != ATTN_OK) return rc;
    const cudaError_t e = launch_fwd_cache_join(p[0], d, st);
    if (e != cudaSuccess) return cuda_fail(e, "join launch");
    return post_launch(s, st);
  }
  if ((rc = cache_maps(mine, few_rows(p[1]), &maps[1])) != ATTN_OK) return rc;
  for (int i = 0; i < 2; ++i)
    if ((rc = launch_cache(maps[i], p[i], d, sms, st)) != ATTN_OK) return rc;
  return post_launch(s, st);
}

}  // extern "C"
