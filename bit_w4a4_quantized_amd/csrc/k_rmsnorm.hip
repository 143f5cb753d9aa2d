// Root-mean-square norm with the residual's addition in front and an 8-bit (or 16-bit) output:
//
//   h = rnd(x + r)  (the stream, kept in r's type)        rstd = 1 / sqrt(mean_k h^2 + eps)
//   v = h w,  a = max(max_k |v|, 2^-100)
//   8 bits : code = rnd(v (qmax / a)),  scale = a rstd / qmax       16 bits : y = rnd(v rstd)
//
// rstd is one factor of the whole row, so it cancels in the codes: they depend on exact maxima
// and elementwise fp32 operations only, not on the order of the row sum.
//
// One pass: a row's values stay in registers between the sums and the codes, so each input byte
// is read and each output byte written once.  HBM bounds it for many rows, latency for few.
#include "block_ops.h"

namespace svdq {

namespace {

constexpr float kTiny = 0x1p-100f;           // floor of a row's maximum: a row of zeros gets codes 0, a finite scale

enum Res { RES_NONE = 0, RES_16 = 1, RES_32 = 2 };

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// Sum of squares and maximum over the row's wpr waves, `first` being the first of them in the block.
// Returns whether the sum of any of the block's rows is not finite (one row a wave: of the wave's).
__device__ __forceinline__ bool row_reduce(float& ss, float& mx, int wpr, int first, float (*red)[16]) {
  ss = wave_sum(ss);
  mx = wave_max(mx);
  if (wpr == 1) return !(ss < INFINITY);
  if ((threadIdx.x & 63) == 0) {
    red[0][threadIdx.x >> 6] = ss;
    red[1][threadIdx.x >> 6] = mx;
  }
  __syncthreads();
  ss = 0.f;
  mx = 0.f;
  for (int i = first; i < first + wpr; i++) {
    ss += red[0][i];
    mx = fmaxf(mx, red[1][i]);
  }
  return !((wpr == 2 ? (red[0][0] + red[0][1]) + (red[0][2] + red[0][3]) : ss) < INFINITY);   // two rows, or one
}

// The squares of finite values from 2^64 on pass fp32's range (bf16 and fp32 hold them up to 2^128):
// such a row's values are squared and summed once more, times 2^-80.
constexpr float kDown = 0x1p-80f;
// The sum over the row, for the block's rows at once.
__device__ __forceinline__ float row_sum(float ss, int wpr, int first, float (*red)[16]) {
  ss = wave_sum(ss);
  if (wpr == 1) return ss;
  __syncthreads();                           // everyone has read the first sums
  if ((threadIdx.x & 63) == 0) red[0][threadIdx.x >> 6] = ss;
  __syncthreads();
  ss = 0.f;
  for (int i = first; i < first + wpr; i++) ss += red[0][i];
  return ss;
}

__device__ __forceinline__ uint32_t code_i8(float v) { return (uint32_t)(int)__builtin_rintf(v) & 0xFFu; }

// Stores go around the caches' ordinary replacement: outputs larger than the L2 caches leave room
// for the inputs (4608 x 3072, 16-bit output: 19.9 us against 25.7; loads the same way are slower).
// The types let a row begin at any element.
template <int BYTES, int ALIGN>
struct Wide {
  typedef uint32_t T __attribute__((ext_vector_type(BYTES / 4), aligned(ALIGN)));
};
template <int ALIGN>
__device__ __forceinline__ void stream16(void* p, const void* v) {
  typename Wide<16, ALIGN>::T x;
  __builtin_memcpy(&x, v, 16);
  __builtin_nontemporal_store(x, static_cast<typename Wide<16, ALIGN>::T*>(p));
}

// n <= 8 16-bit values at p (any element alignment) as a 16-byte piece, zeros behind them.
__device__ __forceinline__ uint4 load_piece(const uint16_t* p, int n) {
  uint4 u = make_uint4(0, 0, 0, 0);
  if (n >= 8) {
    __builtin_memcpy(&u, p, 16);
  } else {
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 7; i++) e[i] = i < n ? p[i] : 0u;
    u = make_uint4(e[0] | (e[1] << 16), e[2] | (e[3] << 16), e[4] | (e[5] << 16), e[6]);
  }
  return u;
}
__device__ __forceinline__ void store_piece(uint16_t* p, const uint4& u, int n) {
  if (n >= 8) {
    stream16<2>(p, &u);
  } else {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 7; i++)
      if (i < n) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}
struct F8 {
  float4 a, b;
};
__device__ __forceinline__ F8 load_piece(const float* p, int n) {
  F8 u{};
  if (n >= 8) {
    __builtin_memcpy(&u, p, 32);
  } else {
    float e[8];
#pragma unroll
    for (int i = 0; i < 7; i++) e[i] = i < n ? p[i] : 0.f;
    u = F8{make_float4(e[0], e[1], e[2], e[3]), make_float4(e[4], e[5], e[6], 0.f)};
  }
  return u;
}
__device__ __forceinline__ void store_piece(float* p, const float* f, int n) {
  if (n >= 8) {
    stream16<4>(p, f);
    stream16<4>(p + 4, f + 4);
  } else {
#pragma unroll
    for (int i = 0; i < 7; i++)
      if (i < n) p[i] = f[i];
  }
}
template <bool BF>
__device__ __forceinline__ void unpack(const uint4& u, float* f) { unpack8(u, BF, f); }
template <bool BF>
__device__ __forceinline__ void unpack(const F8& u, float* f) {
  f[0] = u.a.x; f[1] = u.a.y; f[2] = u.a.z; f[3] = u.a.w;
  f[4] = u.b.x; f[5] = u.b.y; f[6] = u.b.z; f[7] = u.b.w;
}

template <bool BF, typename T>
__device__ __forceinline__ float small_squares(const T* h, int n) {
  float f[8], ss = 0.f;
  unpack<BF>(load_piece(h, n), f);
#pragma unroll
  for (int e = 0; e < 8; e++) ss += (f[e] * kDown) * (f[e] * kDown);
  return ss;
}

// The weighted values v of n <= 8 elements from element o of the output, as codes or 16-bit values.
template <bool BF>
__device__ __forceinline__ void store_out(const NormArgs& a, int64_t o, const float* v, float mul, int n) {
  if (a.out_type == T_INT8 || a.out_type == T_E4M3) {
    uint32_t c[2];
    if (a.out_type == T_INT8) {
#pragma unroll
      for (int w = 0; w < 2; w++)
        c[w] = code_i8(v[4 * w] * mul) | (code_i8(v[4 * w + 1] * mul) << 8) | (code_i8(v[4 * w + 2] * mul) << 16) |
               (code_i8(v[4 * w + 3] * mul) << 24);
    } else {
#pragma unroll
      for (int w = 0; w < 2; w++) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * w] * mul, v[4 * w + 1] * mul, 0, false);
        c[w] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * w + 2] * mul, v[4 * w + 3] * mul, lo, true);
      }
    }
    uint8_t* q = static_cast<uint8_t*>(a.out) + o;
    if (n >= 8) {
      __builtin_nontemporal_store(Wide<8, 1>::T{c[0], c[1]}, reinterpret_cast<Wide<8, 1>::T*>(q));
    } else {
#pragma unroll
      for (int i = 0; i < 7; i++)
        if (i < n) q[i] = (uint8_t)(c[i >> 2] >> (8 * (i & 3)));
    }
  } else {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; e++) y[e] = v[e] * mul;
    store_piece(static_cast<uint16_t*>(a.out) + o, pack8(y, BF), n);
  }
}

__device__ __forceinline__ float root(const NormArgs& a, float ss) { return 1.0f / sqrtf(ss / (float)a.K + a.eps); }
// from the squares of values times 2^-80, next to which eps is nothing
__device__ __forceinline__ float root_down(const NormArgs& a, float ss) { return kDown / sqrtf(ss / (float)a.K); }

// The factor of the weighted values, and the row's scale.
__device__ __forceinline__ float row_factor(const NormArgs& a, int64_t r, float rstd, float mx, bool first) {
  if (a.out_type != T_INT8 && a.out_type != T_E4M3) return rstd;
  mx = fmaxf(mx, kTiny);
  const float qmax = a.out_type == T_INT8 ? 127.f : 448.f;
  if (first) a.scales[r] = mx * rstd / qmax;
  return qmax / mx;
}

template <int RES>
struct ResOf {
  typedef uint16_t T;
  typedef uint4 P;
};
template <>
struct ResOf<RES_32> {
  typedef float T;
  typedef F8 P;
};

// A row in registers: wpr waves, V pieces of 8 elements per lane.  All loads go out first.
template <int RES, bool BF, int V>
__global__ void __launch_bounds__(1024) k_rmsnorm(NormArgs a, int wpr) {
  typedef typename ResOf<RES>::T RT;
  typedef typename ResOf<RES>::P RP;
  __shared__ float red[2][16];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), in_block = wave / wpr;
  const int LANES = wpr * 64, lane = (int)threadIdx.x - in_block * LANES;
  const int row = blockIdx.x * (blockDim.x / LANES) + in_block;
  const bool live = row < a.M;
  const int64_t r = live ? row : a.M - 1;    // rows past the end repeat the last one and store nothing
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + r * a.x_stride;
  const RT* res = RES ? static_cast<const RT*>(a.res) + r * a.res_stride : nullptr;
  RT* res_out = RES ? static_cast<RT*>(a.res_out) + r * a.res_out_stride : nullptr;
  uint4 xr[V];
  RP rr[V];
  float v[V][8], w[V][8];
#pragma unroll
  for (int p = 0; p < V; p++) {
    const int i = (p * LANES + lane) * 8;
    xr[p] = make_uint4(0, 0, 0, 0);
    rr[p] = RP{};
    if (i < a.K) {
      xr[p] = load_piece(x + i, a.K - i);
      if (RES) rr[p] = load_piece(res + i, a.K - i);
    }
  }
  if (a.weight_type == T_F32) {
    F8 wr[V];
#pragma unroll
    for (int p = 0; p < V; p++) {
      const int i = (p * LANES + lane) * 8;
      wr[p] = F8{};
      if (i < a.K) wr[p] = load_piece(static_cast<const float*>(a.weight) + i, a.K - i);
    }
#pragma unroll
    for (int p = 0; p < V; p++) unpack<BF>(wr[p], w[p]);
  } else {
    uint4 wr[V];
#pragma unroll
    for (int p = 0; p < V; p++) {
      const int i = (p * LANES + lane) * 8;
      wr[p] = make_uint4(0, 0, 0, 0);
      if (i < a.K) wr[p] = load_piece(static_cast<const uint16_t*>(a.weight) + i, a.K - i);
    }
#pragma unroll
    for (int p = 0; p < V; p++) unpack<BF>(wr[p], w[p]);
  }
  float ss = 0.f, mx = 0.f;
#pragma unroll
  for (int p = 0; p < V; p++) {
    const int i = (p * LANES + lane) * 8;
    unpack<BF>(xr[p], v[p]);
    if (RES) {
      float g[8];
      unpack<BF>(rr[p], g);
#pragma unroll
      for (int e = 0; e < 8; e++) v[p][e] += g[e];
      if constexpr (RES == RES_16) {
        const uint4 u = pack8(v[p], BF);
        unpack<BF>(u, v[p]);
        if (live && i < a.K) store_piece(res_out + i, u, a.K - i);
      } else if constexpr (RES == RES_32) {
        if (live && i < a.K) store_piece(res_out + i, v[p], a.K - i);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; e++) {
      ss += v[p][e] * v[p][e];
      v[p][e] *= w[p][e];
      mx = fmaxf(mx, fabsf(v[p][e]));
    }
  }
  const bool over = row_reduce(ss, mx, wpr, in_block * wpr, red);
  float rstd = root(a, ss);
  if (over) {
    float sd = 0.f;
#pragma unroll 1
    for (int i = lane * 8; i < a.K; i += LANES * 8)        // the lane's own pieces; the stream as just written
      sd += RES ? small_squares<BF>(res_out + i, a.K - i) : small_squares<BF>(x + i, a.K - i);
    sd = row_sum(sd, wpr, in_block * wpr, red);
    if (!(ss < INFINITY)) rstd = root_down(a, sd);
  }
  if (!live) return;
  const float mul = row_factor(a, r, rstd, mx, lane == 0);
#pragma unroll
  for (int p = 0; p < V; p++) {
    const int i = (p * LANES + lane) * 8;
    if (i < a.K) store_out<BF>(a, r * a.K + i, v[p], mul, a.K - i);
  }
}

// A row too long for registers: one workgroup reads it twice (the second time mostly from the
// caches).  With a residual the second read is of the stream just written by the same thread.
template <int RES, bool BF>
__global__ void __launch_bounds__(1024)
k_rmsnorm_long(NormArgs a) {
  typedef typename ResOf<RES>::T RT;
  __shared__ float red[2][16];
  const int64_t r = blockIdx.x;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + r * a.x_stride;
  const RT* res = RES ? static_cast<const RT*>(a.res) + r * a.res_stride : nullptr;
  RT* res_out = RES ? static_cast<RT*>(a.res_out) + r * a.res_out_stride : nullptr;
  auto weigh = [&](float* v, int i) {
    float w[8];
    if (a.weight_type == T_F32) unpack<BF>(load_piece(static_cast<const float*>(a.weight) + i, a.K - i), w);
    else unpack<BF>(load_piece(static_cast<const uint16_t*>(a.weight) + i, a.K - i), w);
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] *= w[e];
  };
  float ss = 0.f, mx = 0.f;
  for (int i = threadIdx.x * 8; i < a.K; i += 8192) {
    float v[8];
    unpack<BF>(load_piece(x + i, a.K - i), v);
    if (RES) {
      float g[8];
      unpack<BF>(load_piece(res + i, a.K - i), g);
#pragma unroll
      for (int e = 0; e < 8; e++) v[e] += g[e];
      if constexpr (RES == RES_16) {
        const uint4 u = pack8(v, BF);
        unpack<BF>(u, v);
        store_piece(res_out + i, u, a.K - i);
      } else if constexpr (RES == RES_32) {
        store_piece(res_out + i, v, a.K - i);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; e++) ss += v[e] * v[e];
    weigh(v, i);
#pragma unroll
    for (int e = 0; e < 8; e++) mx = fmaxf(mx, fabsf(v[e]));
  }
  float rstd;
  if (row_reduce(ss, mx, 16, 0, red)) {
    ss = 0.f;
    for (int i = threadIdx.x * 8; i < a.K; i += 8192)
      ss += RES ? small_squares<BF>(res_out + i, a.K - i) : small_squares<BF>(x + i, a.K - i);
    rstd = root_down(a, row_sum(ss, 16, 0, red));
  } else {
    rstd = root(a, ss);
  }
  const float mul = row_factor(a, r, rstd, mx, threadIdx.x == 0);
  for (int i = threadIdx.x * 8; i < a.K; i += 8192) {
    float v[8];
    if (RES) unpack<BF>(load_piece(res_out + i, a.K - i), v);
    else unpack<BF>(load_piece(x + i, a.K - i), v);
    weigh(v, i);
    store_out<BF>(a, r * a.K + i, v, mul, a.K - i);
  }
}

template <int RES, bool BF, int V>
hipError_t go(const NormArgs& a, hipStream_t s) {
  const int wpr = (a.K + 512 * V - 1) / (512 * V), rows = wpr > 4 ? 1 : 4 / wpr;
  if (!launchable((a.M + rows - 1) / rows, 64 * wpr * rows)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_rmsnorm<RES, BF, V>), dim3((a.M + rows - 1) / rows), dim3(64 * wpr * rows), 0, s, a, wpr);
  return hipGetLastError();
}

template <int RES, bool BF>
hipError_t launch_res(const NormArgs& a, hipStream_t s) {
  // Pieces a lane (16 bytes of x each, with 16 or 32 of the stream): 48 to 64 bytes in flight are
  // enough, more waves cost their reductions and more pieces leave lanes idle in short rows.  In us,
  // 4608 rows, one piece / two / four: no stream, K = 8192 40.5 / 26.5 / 23.3, 2048 11.3 / 10.0 / 10.8;
  // 16-bit stream, 8192 55.2 / 52.5 / 53.2, 5120 40.0 / 33.8 / 34.3; fp32, 3072 29.1 / 30.5 / 31.0.
  // At most 16 waves hold a row.
  if constexpr (RES == RES_NONE) {
    if (a.K <= 2048) return go<RES, BF, 2>(a, s);
  }
  if constexpr (RES == RES_16) {
    if (a.K <= 16384) return go<RES, BF, 2>(a, s);
  }
  if constexpr (RES == RES_32) {
    if (a.K <= 8192) return go<RES, BF, 1>(a, s);
    if (a.K <= 16384) return go<RES, BF, 2>(a, s);
  }
  if (a.K <= 32768) return go<RES, BF, 4>(a, s);
  if (!launchable(a.M, 1024)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_rmsnorm_long<RES, BF>), dim3(a.M), dim3(1024), 0, s, a);
  return hipGetLastError();
}

template <bool BF>
hipError_t launch_type(const NormArgs& a, hipStream_t s) {
  if (!a.res) return launch_res<RES_NONE, BF>(a, s);
  return a.res_type == T_F32 ? launch_res<RES_32, BF>(a, s) : launch_res<RES_16, BF>(a, s);
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t s) {
  return a.x_type == T_BF16 ? launch_type<true>(a, s) : launch_type<false>(a, s);
}

}  // namespace svdq
