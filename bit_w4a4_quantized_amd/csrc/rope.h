// Shared by the kernels that turn queries and keys by their positions (k_rope.hip, k_append.hip).
//
// The angle is the product in fp64: exact for fp32 positions and frequencies (an fp32 product is
// off by 1e-3 radians at position 32768), rounded to 2^-53 for int32 positions past 2^29.
#pragma once
#include "block_ops.h"

namespace svdq {

// Angles are reduced up to this size; larger ones are taken as it (int32 positions reach it only
// with frequencies past 2^17).
constexpr double kMaxAngle = 0x1p48;

// cos and sin of p f.  k quarter turns are taken off the angle, one fma each with pi/2 in two fp64
// parts: the remainder is good to 2^-52, and the quotient's rounding leaves it within 0.03 of
// (-pi/4, pi/4] at 2^48 and closer below.  Taylor polynomials there: the next terms are below
// 2^-24.  The fp64 operations hide behind the loads (4608 tokens of 24 + 24 heads of 128 21.3 us, an
// fp32 reduction good up to 2^20 21.2; one token 4.2 and 4.1).
__device__ __forceinline__ void cos_sin(double p, float f, float* c, float* s) {
  double q = p * (double)f;
  if (__builtin_fabs(q) > kMaxAngle) q = __builtin_copysign(kMaxAngle, q);
  const double k = __builtin_rint(q * 0.63661977236758134);
  double rem = __builtin_fma(-k, 1.5707963267948966, q);
  rem = __builtin_fma(-k, 6.123233995736766e-17, rem);
  const float r = (float)rem;
  const int n = (int)(k - 4.0 * __builtin_floor(0.25 * k));     // k modulo 4
  const float z = r * r;
  float sn = __builtin_fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
  sn = __builtin_fmaf(z, sn, 1.f / 120.f);
  sn = __builtin_fmaf(z, sn, -1.f / 6.f);
  sn = __builtin_fmaf(z * r, sn, r);
  float cs = __builtin_fmaf(z, 1.f / 40320.f, -1.f / 720.f);
  cs = __builtin_fmaf(z, cs, 1.f / 24.f);
  cs = __builtin_fmaf(z, cs, -0.5f);
  cs = __builtin_fmaf(z, cs, 1.f);
  const float a = n & 1 ? sn : cs, b = n & 1 ? cs : sn;
  *c = (n + 1) & 2 ? -a : a;
  *s = n & 2 ? -b : b;
}

// A store around the caches' ordinary replacement (4608 tokens of 24 + 24 heads of 128: 27.1 -> 21.6 us).
__device__ __forceinline__ void stream16(uint16_t* p, const uint4& v) {
  __builtin_nontemporal_store(u32x4_t{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4_t*>(p));
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
// Sum over groups of `lanes` lanes (a power of two, uniform); every lane gets it.
__device__ __forceinline__ float group_sum(float v, int lanes) {
  if (lanes > 1) v += dpp<0xB1>(v);          // quad_perm: lane ^ 1
  if (lanes > 2) v += dpp<0x4E>(v);          // lane ^ 2
  if (lanes > 4) v += dpp<0x141>(v);         // row_half_mirror: the other four of eight
  if (lanes > 8) v += dpp<0x140>(v);         // row_mirror: the other eight of sixteen
  for (int m = 16; m < lanes; m *= 2) v += __shfl_xor(v, m);
  return v;
}

// 1 / sqrt(mean + eps) of a head from its sum of squares.  Squares of bf16 values from 2^64 on pass
// fp32's range; they are then summed of the values times 2^-80, next to which eps is nothing.
constexpr float kDown = 0x1p-80f;
__device__ __forceinline__ float root(const RopeArgs& a, float ss) {
  return __builtin_amdgcn_rsqf(__builtin_fmaf(ss, 1.0f / (float)a.dim, a.eps));
}
__device__ __forceinline__ float small_square(float v) { return (v * kDown) * (v * kDown); }
__device__ __forceinline__ float root_down(const RopeArgs& a, float ss) {
  return kDown * __builtin_amdgcn_rsqf(ss * (1.0f / (float)a.dim));
}

__device__ __forceinline__ void pair_cos_sin(const RopeArgs& a, int64_t pos, int p, float* c, float* s) {
  const int ax = (p >= a.end[0]) + (p >= a.end[1]) + (p >= a.end[2]);   // ends of absent axes are never reached
  const double at = a.pos_float ? (double)static_cast<const float*>(a.positions)[pos + ax]
                                : (double)static_cast<const int*>(a.positions)[pos + ax];
  cos_sin(at, a.inv_freq[p], c, s);
  if (a.inverse) *s = -*s;
}

}  // namespace svdq
