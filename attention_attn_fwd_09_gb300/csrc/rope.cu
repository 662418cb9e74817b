// Rotary positions of Q and K, and the transposed rotation of their gradients.
//
// A pair (a, b) of a head at position p turns by the angle t = p f_j:
//     y_a = m (a cos t - b sin t),   y_b = m (b cos t + a sin t)
// with the pairs (x_j, x_{j + rot/2}) (half-split) or (x_2j, x_2j+1) (interleaved), f_j the
// pair's frequency and m one factor for the rotated part; columns rot .. d-1 pass through.
// The gradient takes the transposed rotation: the same with sin t negated.
//
// Angles: f_j comes in 64 bits (radians per position).  A CTA turns it once into a
// fixed-point number F_j = f_j / 2 pi mod 1 in units of 2^-64 turns; p F_j mod 2^64 is then
// an exact integer product, its upper 32 bits the angle in turns with the whole turns
// already dropped, so position 10^6 is as exact as position 1 and no argument reduction is
// needed (sincospif of a number in [-1, 1), rounded from these bits by at most 2^-25 half turns, 9.4e-8
// rad).  fp32 p f_j would be wrong by 0.06 rad there.
//
// Bound by bytes (2 read and 2 written per element).  A CTA takes a tile of tokens of one
// sequence and every head of them: the cosines and sines are computed once per token into
// shared memory and used by all heads of Q and K.  The first rows are loaded before they are
// computed.  4 x 2048 tokens of 16 + 16 heads, d = 128: 24.7 us, 5.4 TB/s; the gradient of 2 x 8192
// tokens of 32 + 8 heads: 54.3 us, 6.1 TB/s; a token each of 8 sequences: 2.3 us in a graph.  Few heads
// leave threads idle: 65536 tokens of 1 + 1 heads 38 us, 1.8 TB/s, of 4 + 4 51 us, 5.3 TB/s.
#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kRopeThreads = 256;

// V bf16 values (V = 8, 4, 1) as 32-bit words / one half word.
template <int V>
struct BfVec {
  uint32_t w[V / 2];
};
template <>
struct BfVec<1> {
  uint16_t w[1];
};
template <int V>
__device__ __forceinline__ BfVec<V> ld_vec(const uint16_t* p) {
  BfVec<V> r;
  if constexpr (V == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    r.w[0] = u.x; r.w[1] = u.y; r.w[2] = u.z; r.w[3] = u.w;
  } else if constexpr (V == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    r.w[0] = u.x; r.w[1] = u.y;
  } else {
    r.w[0] = *p;
  }
  return r;
}
template <int V>
__device__ __forceinline__ void st_vec(uint16_t* p, const BfVec<V>& r) {
  if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  else if constexpr (V == 4) *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
  else *p = r.w[0];
}
template <int V>
__device__ __forceinline__ void unpack(const BfVec<V>& r, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = __uint_as_float(uint32_t(r.w[0]) << 16);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      f[2 * i] = __uint_as_float(r.w[i] << 16);
      f[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
    }
  }
}
template <int V>
__device__ __forceinline__ BfVec<V> pack(const float (&f)[V]) {
  BfVec<V> r;
  if constexpr (V == 1) {
    r.w[0] = (uint16_t)(pack_bf16x2(f[0], 0.f) & 0xffffu);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r.w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  }
  return r;
}

// A work item is 2 V elements of one head row: half-split columns j .. j+V-1 with their
// partners at + rot/2, interleaved columns c .. c+2V-1, or 2 V columns of the part that
// passes through.  V = 8 needs rot % 16 == 0 and 16-byte rows, V = 4 rot % 8 == 0 and 8-byte
// rows; V = 1 takes every even rot and alignment.
template <int V, bool INTER, int D>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  extern __shared__ __align__(16) float2 cs[];                       // [tokens][rot / 2] (m cos, m sin)
  constexpr int UPR = D / (2 * V);                     // items per head row
  constexpr int BATCH = 2;                             // items a thread has in flight
  const int half = p.rot / 2;
  unsigned long long* turn = reinterpret_cast<unsigned long long*>(cs + (half << p.tile_shift));   // [rot / 2]
  const int b = blockIdx.x / p.tiles, n0 = (blockIdx.x - b * p.tiles) << p.tile_shift;
  const int tile = 1 << p.tile_shift, tn = min(tile, p.N - n0);
  const int h0 = blockIdx.y * p.head_group, hn = min(p.head_group, p.Hq + p.Hk - h0);
  const int items = (hn << p.tile_shift) * UPR;
  for (int i0 = threadIdx.x; i0 - (int)threadIdx.x < items; i0 += BATCH * kRopeThreads) {
    BfVec<V> a[BATCH], bb[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int i = i0 + k * kRopeThreads, u = i % UPR, r = i / UPR;
      const int n = r & (tile - 1), h = h0 + (r >> p.tile_shift);
      if (i >= items || n >= tn) continue;
      const bool is_q = h < p.Hq;
      const RopeTensor& t = is_q ? p.q : p.k;
      const uint16_t* src = static_cast<const uint16_t*>(t.in) + b * t.in_b + (is_q ? h : h - p.Hq) * t.in_h + (n0 + n) * t.in_n;
      const bool rotated = INTER ? u * 2 * V < p.rot : u * V < half;
      const int ca = (INTER || !rotated) ? u * 2 * V : u * V;
      a[k] = ld_vec<V>(src + ca);
      bb[k] = ld_vec<V>(src + ((INTER || !rotated) ? ca + V : ca + half));
    }
    if (i0 == (int)threadIdx.x) {
      // The angles, while the first rows are under way.
      for (int j = threadIdx.x; j < half; j += kRopeThreads) {
        const double t = p.inv_freq[j] * 0.15915494309189535;          // turns per position
        turn[j] = __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
      }
      __syncthreads();
      for (int i = threadIdx.x; i < tn * half; i += kRopeThreads) {
        const int n = i / half, j = i - n * half;
        const long long pos = p.positions ? p.positions[(long long)b * p.N + n0 + n] : n0 + n;
        const unsigned long long ph = turn[j] * (unsigned long long)pos;
        float s, c;
        sincospif(__int2float_rn((int)(ph >> 32)) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
        // Pairs 2k, 2k + 1 of all items of a row lie side by side: neighbouring threads' 16-byte reads then
        // touch all banks (pair after pair they met in a quarter of them).
        const int slot = V == 1 ? j : (j % V / 2) * (half / V) * 2 + j / V * 2 + (j & 1);
        cs[n * half + slot] = make_float2(c * p.mscale, s * p.mscale * p.sign);
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int i = i0 + k * kRopeThreads, u = i % UPR, r = i / UPR;
      const int n = r & (tile - 1), h = h0 + (r >> p.tile_shift);
      if (i >= items || n >= tn) continue;
      const bool is_q = h < p.Hq;
      const RopeTensor& t = is_q ? p.q : p.k;
      uint16_t* dst = static_cast<uint16_t*>(t.out) + b * t.out_b + (is_q ? h : h - p.Hq) * t.out_h + (n0 + n) * t.out_n;
      const bool rotated = INTER ? u * 2 * V < p.rot : u * V < half;
      const int ca = (INTER || !rotated) ? u * 2 * V : u * V;
      uint16_t* dst_b = dst + ((INTER || !rotated) ? ca + V : ca + half);
      if (!rotated) {
        st_vec<V>(dst + ca, a[k]);
        st_vec<V>(dst_b, bb[k]);
        continue;
      }
      float x[V], y[V], xo[V], yo[V];
      unpack<V>(a[k], x);
      unpack<V>(bb[k], y);
      float cw[V], sw[V];                              // of the item's V pairs
      if constexpr (V == 1) {
        const float2 w = cs[n * half + u];
        cw[0] = w.x;
        sw[0] = w.y;
      } else {
        const float4* w = reinterpret_cast<const float4*>(cs + n * half) + u;
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          const float4 e = w[j * (half / V)];
          cw[2 * j] = e.x;
          sw[2 * j] = e.y;
          cw[2 * j + 1] = e.z;
          sw[2 * j + 1] = e.w;
        }
      }
      if constexpr (INTER && V > 1) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          xo[2 * j] = x[2 * j] * cw[j] - x[2 * j + 1] * sw[j];
          xo[2 * j + 1] = x[2 * j + 1] * cw[j] + x[2 * j] * sw[j];
          yo[2 * j] = y[2 * j] * cw[V / 2 + j] - y[2 * j + 1] * sw[V / 2 + j];
          yo[2 * j + 1] = y[2 * j + 1] * cw[V / 2 + j] + y[2 * j] * sw[V / 2 + j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          xo[j] = x[j] * cw[j] - y[j] * sw[j];
          yo[j] = y[j] * cw[j] + x[j] * sw[j];
        }
      }
      st_vec<V>(dst + ca, pack<V>(xo));
      st_vec<V>(dst_b, pack<V>(yo));
    }
  }
}

template <int V, bool INTER>
cudaError_t launch_v(const RopeParams& p, dim3 grid, size_t smem, cudaStream_t s) {
  if (p.d == 64) rope_kernel<V, INTER, 64><<<grid, kRopeThreads, smem, s>>>(p);
  else if (p.d == 128) rope_kernel<V, INTER, 128><<<grid, kRopeThreads, smem, s>>>(p);
  else if (p.d == 192) rope_kernel<V, INTER, 192><<<grid, kRopeThreads, smem, s>>>(p);
  else rope_kernel<V, INTER, 256><<<grid, kRopeThreads, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(RopeParams p, int vec, int interleaved, int sms, cudaStream_t s) {
  // Tokens per CTA: 4 when that still gives every SM work (the cosines and sines of a token
  // are then shared by all heads), else one token per CTA and the heads split over CTAs so
  // that each thread has about one item.
  const int upr = p.d / (2 * vec), heads = p.Hq + p.Hk;
  p.tile_shift = (long long)p.B * ((p.N + 3) / 4) >= sms ? 2 : 0;
  p.tiles = (p.N + (1 << p.tile_shift) - 1) >> p.tile_shift;
  p.head_group = p.tile_shift > 0 ? heads : (kRopeThreads + upr - 1) / upr;
  const long long gx = (long long)p.B * p.tiles;
  const int gy = (heads + p.head_group - 1) / p.head_group;
  if (gx > 0x7fffffffLL || gy > 65535) return cudaErrorInvalidValue;
  const size_t smem = ((size_t)(1 << p.tile_shift) + 1) * (p.rot / 2) * sizeof(float2);
  const dim3 grid((unsigned)gx, (unsigned)gy);
  if (vec == 8) return interleaved ? launch_v<8, true>(p, grid, smem, s) : launch_v<8, false>(p, grid, smem, s);
  if (vec == 4) return interleaved ? launch_v<4, true>(p, grid, smem, s) : launch_v<4, false>(p, grid, smem, s);
  return interleaved ? launch_v<1, true>(p, grid, smem, s) : launch_v<1, false>(p, grid, smem, s);
}

}  // namespace attn
