// Matrix product with bias, activation and residual in its epilogue:
//
//   y[m, n] = rnd( act( (sum_k x[m, k] w[n, k]) xs[m] ws[n] + b[n] ) + res[m, n] )
//
// for int8 (exact int32 sums), FP8 E4M3, fp16 and bf16 operands (fp32 sums), both row-major
// with K contiguous.  The kernels see rows of bytes: a lane's MFMA operand is one 16-byte piece
// of its row (two for FP8), whatever the type, so staging and layout are the same for all four.
//
// Tiles: four waves in 2 x 2, each TI x TJ MFMA tiles of 32 x 32.  K advances 128 bytes a stage
// through two LDS buffers filled by LDS-DMA one stage ahead.  A row's 128 bytes of a stage are
// eight 16-byte pieces; piece p of row r sits in slot p ^ (r % 8), so the reads of eight
// consecutive rows hit distinct banks and the loads still take whole 128-byte lines.
#include "block_ops.h"
#include "gemm_skel.h"

namespace svdq {

namespace {

using skel::dma16;

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int BK = 128;                      // bytes of K a stage
constexpr uint32_t kPast = 0x80000000u;      // an offset past every resource's range: loads give zeros

template <int TYPE>
struct Mma {
  using Acc = v16f;
};
template <>
struct Mma<T_INT8> {
  using Acc = v16i;
};

// FP8: the matrix core adds eight products at a time, aligned to the largest of the eight with 13
// bits below it (found with one large and several small products; v_mfma_f32_32x32x16_fp8_fp8
// does the same), and the eights' sums in fp32.  The codes themselves carry 3 bits, so the lost
// bits are far below theirs; converting to fp16 first would keep them at half the rate.
//
// acc += the products of two 16-byte pieces per operand (64 bytes of K with the lanes' other half).
template <int TYPE>
__device__ __forceinline__ void mma2(const uint4 (&w)[2], const uint4 (&x)[2], typename Mma<TYPE>::Acc& acc) {
  if constexpr (TYPE == T_INT8) {
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(as_i4(w[0]), as_i4(x[0]), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(as_i4(w[1]), as_i4(x[1]), acc, 0, 0, 0);
  } else if constexpr (TYPE == T_E4M3) {
    const v8i a = {(int)w[0].x, (int)w[0].y, (int)w[0].z, (int)w[0].w, (int)w[1].x, (int)w[1].y, (int)w[1].z, (int)w[1].w};
    const v8i b = {(int)x[0].x, (int)x[0].y, (int)x[0].z, (int)x[0].w, (int)x[1].x, (int)x[1].y, (int)x[1].z, (int)x[1].w};
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, 0, 0, 0, 0, 0, 0);   // scales 0: the unscaled form
  } else if constexpr (TYPE == T_F16) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(w[0]), as_h8(x[0]), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(w[1]), as_h8(x[1]), acc, 0, 0, 0);
  } else {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, w[0]), __builtin_bit_cast(v8bf, x[0]), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, w[1]), __builtin_bit_cast(v8bf, x[1]), acc, 0, 0, 0);
  }
}

__device__ __forceinline__ float activate(float v, int act) {
  if (act == ACT_GELU) return gelu_div(v, 1.0f);
  if (act == ACT_SILU) return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * v));
  return v;
}

// What the kernels take, with strides and K in bytes.
struct Args {
  const uint8_t* x; int64_t x_stride; const float* xs; const uint8_t* w; const float* ws;
  const void* bias; const void* res; int64_t res_stride;
  int M, N, KB, act, bf, wide;               // bf: 16-bit output is bf16; wide: 16-byte pieces of y and res
  void* y; int64_t y_stride;
};

template <int TYPE, int TI, int TJ>
__global__ void __launch_bounds__(256, 2) k_gemm_act(Args a) {
  constexpr int BM = 64 * TI, BN = 64 * TJ;
  constexpr int PX = BM / 32, PW = BN / 32;  // LDS-DMA instructions (8 rows each) per wave and stage
  constexpr int BUF = (BM + BN) * BK;
  constexpr int YS = TJ * 32 * 4 + 16;       // output staging: bytes per row of a wave's 32 x (32 TJ) fp32 block
  static_assert(4 * 32 * YS + 8 * BN <= 2 * BUF, "the epilogue must fit the stage buffers");
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * BUF];
  using Acc = typename Mma<TYPE>::Acc;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int h = lane >> 5, r32 = lane & 31, wm = wave >> 1, wn = wave & 1;
  const int tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + BN - 1) / BN;
  int tm, tn;
  skel::tile_of(blockIdx.x, tiles_m * tiles_n, tiles_m, tiles_n, &tm, &tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int mrows = min(BM, a.M - m0), nrows = min(BN, a.N - n0);
  const rsrc_t rx = make_rsrc(a.x + (int64_t)m0 * a.x_stride, (size_t)((mrows - 1) * a.x_stride + a.KB));
  const rsrc_t rw = make_rsrc(a.w + (int64_t)n0 * a.KB, (size_t)nrows * a.KB);
  const int piece = (lane & 7) ^ (lane >> 3);          // the piece this lane moves: slot lane % 8 of row lane / 8
  uint32_t vx[PX], vw[PW];
#pragma unroll
  for (int i = 0; i < PX; i++)
    vx[i] = (uint32_t)min((wave * PX + i) * 8 + (lane >> 3), mrows - 1) * (uint32_t)a.x_stride + 16u * piece;
#pragma unroll
  for (int i = 0; i < PW; i++)
    vw[i] = (uint32_t)min((wave * PW + i) * 8 + (lane >> 3), nrows - 1) * (uint32_t)a.KB + 16u * piece;
  auto load = [&](int k0, uint8_t* buf) {
    const bool past = k0 + 16 * piece >= a.KB;         // pieces past the end of K read as zeros
#pragma unroll
    for (int i = 0; i < PX; i++) dma16(rx, buf + (wave * PX + i) * 1024, past ? kPast : vx[i], (uint32_t)k0);
#pragma unroll
    for (int i = 0; i < PW; i++) dma16(rw, buf + BM * BK + (wave * PW + i) * 1024, past ? kPast : vw[i], (uint32_t)k0);
  };
  Acc acc[TJ][TI];
#pragma unroll
  for (int tj = 0; tj < TJ; tj++)
#pragma unroll
    for (int ti = 0; ti < TI; ti++)
#pragma unroll
      for (int i = 0; i < 16; i++) acc[tj][ti][i] = 0;
  const int stages = (a.KB + BK - 1) / BK;
  load(0, lds);
  for (int st = 0; st < stages; st++) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();                         // stage st is in; everyone has read stage st - 1
    if (st + 1 < stages) load((st + 1) * BK, lds + ((st + 1) & 1) * BUF);
    const uint8_t* b = lds + (st & 1) * BUF;
#pragma unroll
    for (int ks = 0; ks < 2; ks++) {
      uint4 xf[TI][2], wf[TJ][2];
#pragma unroll
      for (int j = 0; j < 2; j++) {
        const int p = 4 * ks + 2 * j + h;
#pragma unroll
        for (int ti = 0; ti < TI; ti++) {
          const int r = (wm * TI + ti) * 32 + r32;
          xf[ti][j] = *reinterpret_cast<const uint4*>(b + r * BK + 16 * (p ^ (r & 7)));
        }
#pragma unroll
        for (int tj = 0; tj < TJ; tj++) {
          const int r = (wn * TJ + tj) * 32 + r32;
          wf[tj][j] = *reinterpret_cast<const uint4*>(b + BM * BK + r * BK + 16 * (p ^ (r & 7)));
        }
      }
#pragma unroll
      for (int tj = 0; tj < TJ; tj++)
#pragma unroll
        for (int ti = 0; ti < TI; ti++) mma2<TYPE>(wf[tj], xf[ti], acc[tj][ti]);
    }
  }
  __syncthreads();                           // the stage buffers become the epilogue's
  // lane (r32, h) holds row ti*32 + r32 and columns tj*32 + 8 q + 4 h + j of its wave's block
  float* cs = reinterpret_cast<float*>(lds + 4 * 32 * YS);   // column scales and bias, BN each
  for (int i = threadIdx.x; i < BN; i += 256) {
    const int n = n0 + i;
    cs[i] = a.ws && n < a.N ? a.ws[n] : 1.f;
    cs[BN + i] = a.bias && n < a.N ? load16(a.bias, n, a.bf) : 0.f;
  }
  __syncthreads();
  uint8_t* ys = lds + wave * 32 * YS;
#pragma unroll
  for (int ti = 0; ti < TI; ti++) {
    const int mb = m0 + (wm * TI + ti) * 32, nb = n0 + wn * TJ * 32;
    const float sx = a.xs ? a.xs[min(mb + r32, a.M - 1)] : 1.f;
#pragma unroll
    for (int tj = 0; tj < TJ; tj++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int c = tj * 32 + 8 * q + 4 * h;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; j++)
          v[j] = activate((float)acc[tj][ti][4 * q + j] * sx * cs[wn * TJ * 32 + c + j] + cs[BN + wn * TJ * 32 + c + j], a.act);
        *reinterpret_cast<float4*>(ys + r32 * YS + c * 4) = make_float4(v[0], v[1], v[2], v[3]);
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (a.wide) {
      constexpr int PR = TJ * 4;             // 8-column pieces per row
      for (int i = lane; i < 32 * PR; i += 64) {
        const int r = i / PR, c = (i % PR) * 8, m = mb + r, n = nb + c;
        if (m >= a.M || n >= a.N) continue;
        float v[8];
        *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(ys + r * YS + c * 4);
        *reinterpret_cast<float4*>(v + 4) = *reinterpret_cast<const float4*>(ys + r * YS + c * 4 + 16);
        if (a.res) {
          float g[8];
          unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.res) + m * a.res_stride + n), a.bf, g);
#pragma unroll
          for (int e = 0; e < 8; e++) v[e] += g[e];
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + m * a.y_stride + n) = pack8(v, a.bf);
      }
    } else {
      for (int i = lane; i < 32 * TJ * 32; i += 64) {
        const int r = i / (TJ * 32), c = i % (TJ * 32), m = mb + r, n = nb + c;
        if (m >= a.M || n >= a.N) continue;
        float v = *reinterpret_cast<const float*>(ys + r * YS + c * 4);
        if (a.res) v += load16(a.res, m * a.res_stride + n, a.bf);
        store16(a.y, m * a.y_stride + n, v, a.bf);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

template <int TYPE, int TI, int TJ>
hipError_t go(const Args& a, hipStream_t s) {
  const int64_t tiles = (int64_t)((a.M + 64 * TI - 1) / (64 * TI)) * ((a.N + 64 * TJ - 1) / (64 * TJ));
  hipLaunchKernelGGL((k_gemm_act<TYPE, TI, TJ>), dim3((unsigned)tiles), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int TYPE>
hipError_t launch_type(const Args& a, hipStream_t s) {
  const int64_t big = (int64_t)((a.M + 127) / 128) * ((a.N + 127) / 128);
  return big >= 256 ? go<TYPE, 2, 2>(a, s) : go<TYPE, 1, 1>(a, s);
}

}  // namespace

hipError_t launch_gemm_act(const GemmActArgs& g, hipStream_t s) {
  const int eb = g.type == T_F16 || g.type == T_BF16 ? 2 : 1;
  auto vec = [](const void* p, int64_t stride) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && stride % 8 == 0; };
  Args a{};
  a.x = static_cast<const uint8_t*>(g.x);
  a.x_stride = g.x_stride * eb;
  a.xs = g.xs;
  a.w = static_cast<const uint8_t*>(g.w);
  a.ws = g.ws;
  a.bias = g.bias;
  a.res = g.res;
  a.res_stride = g.res_stride;
  a.M = g.M;
  a.N = g.N;
  a.KB = g.K * eb;
  a.act = g.act;
  a.bf = g.out_type == T_BF16;
  a.wide = g.N % 8 == 0 && vec(g.y, g.y_stride) && (!g.res || vec(g.res, g.res_stride));
  a.y = g.y;
  a.y_stride = g.y_stride;
  switch (g.type) {
    case T_INT8: return launch_type<T_INT8>(a, s);
    case T_E4M3: return launch_type<T_E4M3>(a, s);
    case T_F16: return launch_type<T_F16>(a, s);
    case T_BF16: return launch_type<T_BF16>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace svdq
