// Angles of rotary positions in turns, as fixed-point numbers (rope.cu, rope_append.cu).
#pragma once
#include <cstdint>

namespace attn {

// Radians per position (fp64) -> turns per position modulo 1, in units of 2^-64.
__device__ __forceinline__ unsigned long long turns_per_position(double inv_freq) {
  const double t = inv_freq * 0.15915494309189535;
  return __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
}

// Sine and cosine of `pos` times that: the product drops whole turns, its upper 32 bits are the angle.
__device__ __forceinline__ void turn_sincos(unsigned long long turn, long long pos, float& s, float& c) {
  const unsigned long long ph = turn * (unsigned long long)pos;
  sincospif(__int2float_rn((int)(ph >> 32)) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
}

// The same with the nearest quarter turn taken out before the angle is rounded to fp32: off by 2.5e-8 rad
// instead of 9.4e-8.  For values that are rounded once only, to 8 bits: of 16.8 million codes 12 are not the
// nearest ones, as with sines and cosines rounded from 64 bits (15).
__device__ __forceinline__ void turn_sincos_near(unsigned long long turn, long long pos, float& s, float& c) {
  const uint32_t at = (uint32_t)(turn * (unsigned long long)pos >> 32), quarter = (at + 0x20000000u) >> 30;
  float a, b;
  sincospif(__int2float_rn((int)(at - (quarter << 30))) * 4.656612873077393e-10f, &a, &b);   // within +-1/4
  s = quarter & 1 ? b : a;
  c = quarter & 1 ? -a : b;
  if (quarter & 2) {
    s = -s;
    c = -c;
  }
}

// A pair (a, b) turned: x = a c - b s, y = b c + a s.  Which product is rounded by itself is written down, so that
// all kernels turn a pair to the same bits.
__device__ __forceinline__ void turn_pair(float a, float b, float c, float s, float& x, float& y) {
  x = __fmaf_rn(a, c, -__fmul_rn(b, s));
  y = __fmaf_rn(b, c, __fmul_rn(a, s));
}
// One of the two: x turned, z its partner.
__device__ __forceinline__ float turn_one(float x, float z, float c, float s, bool second) {
  return __fmaf_rn(x, c, __fmul_rn(second ? z : -z, s));
}

}  // namespace attn
