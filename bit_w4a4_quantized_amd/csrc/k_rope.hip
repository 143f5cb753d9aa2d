// Rotary positions with several axes (time, height, width), with the heads' RMS norm in front:
//
//   u = x w / sqrt(mean_d x^2 + eps)   (u = x without a weight)
//   angle[t, p] = position[t, axis(p)] f[p];  (u_i, u_j) -> (u_i cos - u_j sin, u_i sin + u_j cos)
//
// for the pair p of elements (i, j): adjacent (2p, 2p + 1) or half apart (p, p + pairs).  Elements
// past 2 pairs pass through.  `inverse` turns by the opposite angle, which is also the gradient
// with respect to u.  HBM bounds it: every value is read once and written once; cosines and sines
// are computed once per token and pair and shared by the token's heads.
//
// The angle is the exact product: its fp32 rounding is 2^-25 of the angle, 1e-3 radians at position
// 32768.  The product and its rounding error (one fma) are reduced to (-pi, pi] before sine and cosine.
#include "block_ops.h"

namespace svdq {

namespace {

// cos and sin of p f: q + e is the exact product, and k whole turns are taken off q in three
// steps, 2 pi being 6.28125 (8 bits: its multiples cancel exactly against q for k < 2^16), the
// fp32 rest and the rest's own error.
__device__ __forceinline__ void cos_sin(float p, float f, float* c, float* s) {
  const float q = p * f, e = __builtin_fmaf(p, f, -q);
  const float k = __builtin_rintf(q * 0.15915494309189535f);
  float r = __builtin_fmaf(-k, 6.28125f, q);
  r = __builtin_fmaf(-k, 0.00193530716933310031890869f, r);
  r = __builtin_fmaf(-k, 1.0253376e-11f, r) + e;
  *c = cosf(r);
  *s = sinf(r);
}

// One wave per (batch, token, head): lanes stride over the pairs and the elements behind them.
__global__ void __launch_bounds__(256) k_rope_plain(RopeArgs a, int64_t units) {
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (unit >= units) return;
  const int lane = threadIdx.x & 63;
  const int heads = a.op[0].heads + (a.nops > 1 ? a.op[1].heads : 0);
  int hd = (int)(unit % heads);
  const int64_t bt = unit / heads;
  const int64_t t = bt % a.tokens, b = bt / a.tokens;
  const RopeOperand& o = hd < a.op[0].heads ? a.op[0] : a.op[1];
  if (hd >= a.op[0].heads) hd -= a.op[0].heads;
  const uint16_t* in = static_cast<const uint16_t*>(o.in) + b * o.in_batch + t * o.in_token + hd * o.in_head;
  uint16_t* out = static_cast<uint16_t*>(o.out) + b * o.out_batch + t * o.out_token + hd * o.out_head;
  const bool bf = a.type == T_BF16;
  float rstd = 1.f;
  if (o.weight) {
    float ss = 0.f;
    for (int d = lane; d < a.dim; d += 64) {
      const float v = load16(in, d, bf);
      ss += v * v;
    }
    for (int m = 32; m > 0; m >>= 1) ss += __shfl_xor(ss, m);
    rstd = 1.0f / sqrtf(ss / (float)a.dim + a.eps);
  }
  auto val = [&](int d) {
    const float v = load16(in, d, bf);
    return o.weight ? v * rstd * o.weight[d] : v;
  };
  const int64_t pos = b * a.pos_batch + t * a.pos_token;
  for (int p = lane; p < a.pairs; p += 64) {
    int ax = 0;
    while (p >= a.end[ax]) ax++;
    const float at = a.pos_float ? static_cast<const float*>(a.positions)[pos + ax]
                                 : (float)static_cast<const int*>(a.positions)[pos + ax];
    float c, s;
    cos_sin(at, a.inv_freq[p], &c, &s);
    if (a.inverse) s = -s;
    const int i = a.halves ? p : 2 * p, j = a.halves ? p + a.pairs : 2 * p + 1;
    const float u = val(i), w = val(j);
    store16(out, i, u * c - w * s, bf);
    store16(out, j, u * s + w * c, bf);
  }
  for (int d = 2 * a.pairs + lane; d < a.dim; d += 64) store16(out, d, val(d), bf);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t s) {
  const int64_t units = (int64_t)a.batch * a.tokens * (a.op[0].heads + (a.nops > 1 ? a.op[1].heads : 0));
  hipLaunchKernelGGL(k_rope_plain, dim3((unsigned)((units + 3) / 4)), dim3(256), 0, s, a, units);
  return hipGetLastError();
}

}  // namespace svdq
