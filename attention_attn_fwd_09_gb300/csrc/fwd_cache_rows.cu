// Attention of packed queries over a paged e4m3 cache: any number of rows, the plain kernel.
//
// O_i = sum_j softmax_j(scale q_i . k_j sk) v_j sv over the keys j <= i + len - n (causal) or
// j < len; one warp per query row and head, 32 keys at a time with a running maximum and sum.
#include <cstdint>

#include "cache.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace attn {
namespace {

template <int D>
__global__ void __launch_bounds__(128) fwd_cache_simple_kernel(const CacheParams p) {
  __shared__ float qs[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x;
  int b = -1;
  bool bad = false;
  for (int base = 0; base < p.B; base += 128) {
    const int i = base + threadIdx.x;
    bool below = false, wrong = false;
    if (i < p.B) {
      const int c0 = p.cu_q[i], c1 = p.cu_q[i + 1], len = p.kv_lens[i];
      wrong = c1 < c0 || c0 < 0 || c1 - c0 > p.max_q || len < 0 || len > p.max_len || (p.causal && c1 - c0 > len) ||
              (i == 0 && c0 != 0) || (i == p.B - 1 && c1 != p.total_q);
      below = c0 <= t;
    }
    bad |= __syncthreads_or(wrong) != 0;
    b += __syncthreads_count(below);
  }
  if (bad) {
    if (threadIdx.x == 0) atomicExch(p.status, DEV_BAD_OFFSETS);
    return;
  }
  const int n = p.cu_q[b + 1] - p.cu_q[b], len = p.kv_lens[b];
  const int vis = p.causal ? t - p.cu_q[b] + len - n + 1 : len;
  for (int h = blockIdx.y * 4 + warp; h < p.Hq; h += gridDim.y * 4) {
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + ((long long)h * p.total_q + t) * D;
    for (int c = lane; c < D; c += 32) qs[warp][c] = __uint_as_float(uint32_t(q[c]) << 16);
    __syncwarp();
    const int hk = h / p.g;
    float m = -INFINITY, l = 0.f, o[D / 32];
    for (int c = 0; c < D / 32; ++c) o[c] = 0.f;
    for (int k0 = 0; k0 < vis; k0 += 32) {
      const int key = k0 + lane;
      float s = -INFINITY, sv = 0.f;
      const uint8_t* vrow = nullptr;
      if (key < vis) {
        const int page = p.table[(long long)b * p.max_pages + key / p.page];
        if (page < 0 || page >= p.num_pages) {
          atomicExch(p.status, DEV_BAD_PAGE);
        } else {
          const long long ph = (long long)page * p.Hkv + hk;
          const long long row = (ph * p.page + key % p.page) * D;
          vrow = p.v_cache + row;
          sv = p.v_scale[ph];
          float acc = 0.f;
          for (int c = 0; c < D; c += 4) {
            float x0, x1, x2, x3;
            e4m3x4_to_f32(*reinterpret_cast<const uint32_t*>(p.k_cache + row + c), x0, x1, x2, x3);
            acc += qs[warp][c] * x0 + qs[warp][c + 1] * x1 + qs[warp][c + 2] * x2 + qs[warp][c + 3] * x3;
          }
          s = acc * (p.k_scale[ph] * p.c);
        }
      }
      float mx = s;
      for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, x));
      const float mn = fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn;
      const float alpha = exp2f(m - mu), e = exp2f(s - mu);
      float sum = e;
      for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(~0u, sum, x);
      l = l * alpha + sum;
      m = mn;
      for (int c = 0; c < D / 32; ++c) o[c] *= alpha;
      for (int k = 0; k < 32; ++k) {
        const float w = __shfl_sync(~0u, e * sv, k);
        const uint8_t* vr = reinterpret_cast<const uint8_t*>(__shfl_sync(~0u, (unsigned long long)vrow, k));
        if (vr == nullptr) continue;
        for (int c = 0; c < D / 32; ++c) {
          const uint32_t f = e4m3x2_f16x2(vr[c * 32 + lane]);
          o[c] += w * __low2float(*reinterpret_cast<const __half2*>(&f));
        }
      }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint16_t* out = static_cast<uint16_t*>(p.o) + ((long long)h * p.total_q + t) * D;
    for (int c = 0; c < D / 32; ++c) out[c * 32 + lane] = (uint16_t)(pack_bf16x2(o[c] * inv, 0.f) & 0xffffu);
    if (lane == 0) p.lse[(long long)h * p.total_q + t] = (m + log2f(l)) * 0.6931471805599453f;
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_fwd_cache_rows(const CacheParams& p, int d, cudaStream_t s) {
  const dim3 grid((unsigned)p.total_q, (unsigned)((p.Hq + 3) / 4));
  if (d == 64) fwd_cache_simple_kernel<64><<<grid, 128, 0, s>>>(p);
  else fwd_cache_simple_kernel<128><<<grid, 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace attn
