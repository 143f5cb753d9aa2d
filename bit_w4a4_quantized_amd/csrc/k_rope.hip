// Rotary positions with several axes (time, height, width), with the heads' RMS norm in front:
//
//   u = x w / sqrt(mean_d x^2 + eps)   (u = x without a weight)
//   angle[t, p] = position[t, axis(p)] f[p];  (u_i, u_j) -> (u_i cos - u_j sin, u_i sin + u_j cos)
//
// for the pair p of elements (i, j): adjacent (2p, 2p + 1) or half apart (p, p + pairs).  Elements
// past 2 pairs pass through.  `inverse` turns by the opposite angle, which is also the gradient
// with respect to u.  HBM bounds it: every value is read once and written once; cosines and sines
// are computed once per wave, each by one lane, and shared through LDS by the token's heads.
//
// The angle is the product in fp64: exact for fp32 positions and frequencies (an fp32 product is
// off by 1e-3 radians at position 32768), rounded to 2^-53 for int32 positions past 2^29.
#include "block_ops.h"

namespace svdq {

namespace {

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

// 16-byte pieces: `lanes` lanes (a power of two) hold a head, lane j its pieces j and j + half of
// eight values, so a wave has 64 / lanes lane groups and takes U units (heads of tokens) per
// group, all loads in flight.  An operand of many heads gives a wave one of `batches` parts of a
// token's heads; one of few heads gives it all heads of `tw` tokens.
struct Split {
  int tw, batches;
  int waves;                                 // of the operand
  uint32_t magic;                            // ceil(2^32 / heads): unit / heads for units below 2^16; 0 for one head
};
struct Splits {
  Split of[2];
  uint32_t share;                            // of the second operand's workgroups among all, times 2^32, rounded up
};

// Pairs of neighbours over the whole head or behind which values stay unturned, or half apart (whole
// heads).  A form of its own for the second costs the others nothing (5 registers and 1% if tested in one).
enum Form { ADJACENT, PARTIAL, HALVES };

template <bool BF, Form FORM, int U>
__global__ void __launch_bounds__(256) k_rope(RopeArgs a, int lanes, Splits sp) {
  __shared__ __attribute__((aligned(16))) float table[4][2][512];   // cosines and sines of each wave's tokens
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  // workgroups of the two operands in even turns: a token's queries and keys are read at about the
  // same time (2 x 16384 tokens of a packed projection took 4% longer with all queries first)
  const uint32_t k1 = __umulhi(blockIdx.x, sp.share);
  const int which = __umulhi(blockIdx.x + 1, sp.share) > k1;
  const int id = __builtin_amdgcn_readfirstlane((int)(which ? k1 : blockIdx.x - k1) * 4 + wave);
  const Split& w_ = sp.of[which];
  if (id >= w_.waves) return;                // whole waves; no workgroup barrier below
  const RopeOperand& o = a.op[which];
  const int groups = 64 / lanes, j = lane % lanes, g = lane / lanes;
  const int nv = a.dim / 8, half = (nv + 1) / 2, pairs = a.dim / 2;
  const bool in0 = j < half, in1 = j + half < nv;
  const int part = id % w_.batches, tok = id / w_.batches * w_.tw;   // first token, over the batch
  const int b0 = tok / a.tokens, t0 = tok - b0 * a.tokens;
  const int nt = min(w_.tw, a.batch * a.tokens - tok);
  const int first = part * U * groups, last = min(nt * o.heads, first + U * groups);
  uint4 raw[U][2];
  uint16_t* out[U];
  int tl[U];
#pragma unroll
  for (int i = 0; i < U; i++) {
    const int u = first + i * groups + g;
    raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
    out[i] = nullptr;
    tl[i] = 0;
    if (u < last) {
      int hd = u, b = b0, t = t0;
      if (w_.tw > 1) {
        tl[i] = w_.magic ? (int)__umulhi((uint32_t)u, w_.magic) : u;
        hd = u - tl[i] * o.heads;
        t += tl[i];
        while (t >= a.tokens) {
          t -= a.tokens;
          b++;
        }
      }
      const uint16_t* p = static_cast<const uint16_t*>(o.in) + b * o.in_batch + t * o.in_token + hd * o.in_head;
      out[i] = static_cast<uint16_t*>(o.out) + b * o.out_batch + t * o.out_token + hd * o.out_head;
      if (in0) raw[i][0] = *reinterpret_cast<const uint4*>(p + j * 8);
      if (in1) raw[i][1] = *reinterpret_cast<const uint4*>(p + (j + half) * 8);
    }
  }
  // pairs past the turned ones get the identity (not used: below)
  for (int i = lane; i < nt * pairs; i += 64) {
    const int tl_ = w_.tw > 1 ? i / pairs : 0, p = i - tl_ * pairs;
    int b = b0, t = t0 + tl_;
    while (t >= a.tokens) {
      t -= a.tokens;
      b++;
    }
    float c = 1.f, s = 0.f;
    if (p < a.pairs) pair_cos_sin(a, b * a.pos_batch + t * a.pos_token, p, &c, &s);
    table[wave][0][i] = c;
    table[wave][1][i] = s;
  }
  const bool norm = o.weight != nullptr;
  float w[2][8];
  if (norm) {
#pragma unroll
    for (int v = 0; v < 2; v++) __builtin_memcpy(w[v], o.weight + min((j + v * half) * 8, a.dim - 8), 32);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < U; i++) {
    float u[2][8], c[8], s[8], y[2][8];
    unpack8(raw[i][0], BF, u[0]);
    unpack8(raw[i][1], BF, u[1]);
    // the lane's eight pairs: of its two pieces (adjacent), or between them (half apart)
#pragma unroll
    for (int v = 0; v < 2; v++) {
      const int p = tl[i] * pairs + min(FORM == HALVES ? j * 8 + v * 4 : (j + v * half) * 4, pairs - 4);
      *reinterpret_cast<float4*>(c + 4 * v) = *reinterpret_cast<const float4*>(&table[wave][0][p]);
      *reinterpret_cast<float4*>(s + 4 * v) = *reinterpret_cast<const float4*>(&table[wave][1][p]);
    }
    if (norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; e++) ss += u[0][e] * u[0][e] + u[1][e] * u[1][e];
      ss = group_sum(ss, lanes);
      float rstd = root(a, ss);
      if (BF && __any(!(ss < INFINITY))) {   // the whole wave, for the sum's lanes
        float sd = 0.f;
#pragma unroll
        for (int e = 0; e < 8; e++) sd += small_square(u[0][e]) + small_square(u[1][e]);
        sd = group_sum(sd, lanes);
        if (!(ss < INFINITY)) rstd = root_down(a, sd);
      }
#pragma unroll
      for (int v = 0; v < 2; v++)
#pragma unroll
        for (int e = 0; e < 8; e++) u[v][e] = u[v][e] * rstd * w[v][e];
    }
    if (FORM == HALVES) {
#pragma unroll
      for (int e = 0; e < 8; e++) {
        y[0][e] = u[0][e] * c[e] - u[1][e] * s[e];
        y[1][e] = u[0][e] * s[e] + u[1][e] * c[e];
      }
    } else {
#pragma unroll
      for (int v = 0; v < 2; v++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float cc = c[4 * v + e], sn = s[4 * v + e];
          y[v][2 * e] = u[v][2 * e] * cc - u[v][2 * e + 1] * sn;
          y[v][2 * e + 1] = u[v][2 * e] * sn + u[v][2 * e + 1] * cc;
        }
    }
    // values behind the pairs as they are: turned by the identity, an infinity or NaN would reach its neighbour
    if (FORM == PARTIAL) {
#pragma unroll
      for (int v = 0; v < 2; v++)
#pragma unroll
        for (int e = 0; e < 8; e++)
          if ((j + v * half) * 4 + e / 2 >= a.pairs) y[v][e] = u[v][e];
    }
    if (out[i]) {
      if (in0) stream16(out[i] + j * 8, pack8(y[0], BF));
      if (in1) stream16(out[i] + (j + half) * 8, pack8(y[1], BF));
    }
  }
}

// Any dim, pairing, stride and alignment: one wave per (batch, token, head), lanes stride over the
// pairs and the elements behind them.
__global__ void __launch_bounds__(256) k_rope_any(RopeArgs a, int64_t units) {
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
  if (o.weight) {                            // every lane's reads are done before the first store below
    float ss = 0.f;
    for (int d = lane; d < a.dim; d += 64) {
      const float v = load16(in, d, bf);
      ss += v * v;
    }
    ss = group_sum(ss, 64);
    rstd = root(a, ss);
    if (!(ss < INFINITY)) {                  // the same in every lane
      float sd = 0.f;
      for (int d = lane; d < a.dim; d += 64) sd += small_square(load16(in, d, bf));
      rstd = root_down(a, group_sum(sd, 64));
    }
  }
  auto val = [&](int d) {
    const float v = load16(in, d, bf);
    return o.weight ? v * rstd * o.weight[d] : v;
  };
  const int64_t pos = b * a.pos_batch + t * a.pos_token;
  for (int p = lane; p < a.pairs; p += 64) {
    float c, s;
    pair_cos_sin(a, pos, p, &c, &s);
    const int i = a.halves ? p : 2 * p, j = a.halves ? p + a.pairs : 2 * p + 1;
    const float u = val(i), w = val(j);
    store16(out, i, u * c - w * s, bf);
    store16(out, j, u * s + w * c, bf);
  }
  for (int d = 2 * a.pairs + lane; d < a.dim; d += 64) store16(out, d, val(d), bf);
}

bool wide(const RopeArgs& a) {
  if (a.dim % 8 || (a.halves && 2 * a.pairs != a.dim) || (a.halves && a.dim % 16)) return false;
  for (int i = 0; i < a.nops; i++) {
    const RopeOperand& o = a.op[i];
    if ((reinterpret_cast<uintptr_t>(o.in) | reinterpret_cast<uintptr_t>(o.out)) & 15u) return false;
    if ((o.in_batch | o.in_token | o.in_head | o.out_batch | o.out_token | o.out_head) % 8) return false;
  }
  return true;
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t s) {
  const int64_t tokens = (int64_t)a.batch * a.tokens;
  if (!wide(a)) {
    const int64_t units = tokens * (a.op[0].heads + (a.nops > 1 ? a.op[1].heads : 0));
    if (!launchable((units + 3) / 4, 256)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(k_rope_any, dim3((unsigned)((units + 3) / 4)), dim3(256), 0, s, a, units);
    return hipGetLastError();
  }
  int lanes = 1;
  while (lanes * 16 < a.dim) lanes *= 2;
  // Three units in flight per lane group for many tokens whose heads waste no more of three than
  // of two (4608 tokens of 24 heads of 128: 21.8 us against 23.6), else two (9000 tokens of 16 heads
  // of 256 59.6 us against 63.0, one token 5.1 and 5.5, launch included)
  const int groups = 64 / lanes;
  auto wasted = [&](int u) {
    int n = 0;
    for (int i = 0; i < a.nops; i++) n += (a.op[i].heads + u * groups - 1) / (u * groups) * u * groups - a.op[i].heads;
    return n;
  };
  const int U = tokens >= 2048 && wasted(3) <= wasted(2) ? 3 : 2;
  const int per = U * groups;                // units a wave
  Splits sp{};
  uint32_t blocks[2] = {0, 0};
  for (int i = 0; i < a.nops; i++) {
    Split& w = sp.of[i];
    const int heads = a.op[i].heads;
    w.batches = (heads + per - 1) / per;
    // all heads of several tokens where they fit a wave and the table, with two waves left per SIMD
    int64_t tw = per / heads < 1024 / a.dim ? per / heads : 1024 / a.dim;
    tw = tw < tokens / 2048 ? tw : tokens / 2048;
    w.tw = tw < 1 ? 1 : (int)tw;
    w.waves = (int)((tokens + w.tw - 1) / w.tw) * w.batches;
    w.magic = heads == 1 ? 0u : (uint32_t)(((1ull << 32) + heads - 1) / heads);
    blocks[i] = (uint32_t)(w.waves + 3) / 4;
  }
  const uint32_t all = blocks[0] + blocks[1];
  if (!launchable(all, 256)) return hipErrorInvalidConfiguration;
  sp.share = (uint32_t)((((uint64_t)blocks[1] << 32) + all - 1) / all);
  const bool bf = a.type == T_BF16;
  const auto two = a.halves            ? (bf ? k_rope<true, HALVES, 2> : k_rope<false, HALVES, 2>)
                   : 2 * a.pairs < a.dim ? (bf ? k_rope<true, PARTIAL, 2> : k_rope<false, PARTIAL, 2>)
                                         : (bf ? k_rope<true, ADJACENT, 2> : k_rope<false, ADJACENT, 2>);
  const auto three = a.halves            ? (bf ? k_rope<true, HALVES, 3> : k_rope<false, HALVES, 3>)
                     : 2 * a.pairs < a.dim ? (bf ? k_rope<true, PARTIAL, 3> : k_rope<false, PARTIAL, 3>)
                                           : (bf ? k_rope<true, ADJACENT, 3> : k_rope<false, ADJACENT, 3>);
  hipLaunchKernelGGL(U == 2 ? two : three, dim3(all), dim3(256), 0, s, a, lanes, sp);
  return hipGetLastError();
}

}  // namespace svdq
