// svdq_gemm_act_residual for few token rows (M <= 64): the weight's bytes bound it.
//
// A workgroup owns 16 weight rows (output columns) and all token rows; its four waves split K in
// turns of 128 bytes and add their sums in LDS, in a fixed order.  Each wave streams its pieces
// through a ring of R stages of its own (LDS-DMA, whole cache lines), so there is no barrier in
// the K loop.  N / 16 workgroups keep the chip loading from N = 3072 on.  The token rows pass
// through the same rings out of the caches; rows past M are zeros that touch no memory.
//
// A row's 128 bytes are eight 16-byte pieces; piece p of row r sits in slot p ^ (r / 2 % 8): the
// reads of sixteen rows at one piece hit distinct banks.  v_mfma 16 x 16: lane (r16, q) holds
// pieces q and 4 + q of its row, and gets columns 4 q ... 4 q + 3 of token row r16.
//
// The rings are short, so that two or three workgroups share a CU: with R = 4 and one or two of
// them 16 x 3072 x 12288 (M x K x N) in int8 took 11.4 us, 9.2 with R = 3; 64 rows 20.9, 14.5 with R = 2.
// 1 x 12288 x 3072 takes 9.1 us in int8 (13.3 in split 64 x 64 tiles), 9.6 in E4M3 with its conversion to
// fp16 and 13.9 in bf16; 1 x 3072 x 12288 8.9, 9.1 and 13.8 (tiles 10.7, 12.0 and 16.2): 4.1 ... 5.5
// TB/s of weight.  With 33 rows and more the token rows' traffic (each workgroup reads them all)
// passes the weight's, and wide products go to tiles.
#include "gemm_act.h"

namespace svdq {
namespace gact {

namespace {

template <int TYPE>
struct Mma {
  using Acc = v4f;
};
template <>
struct Mma<T_INT8> {
  using Acc = v4i;
};

// A piece's MFMA operands: one, or for E4M3 its two halves in fp16.
template <int TYPE>
struct Frag {
  uint4 v[TYPE == T_E4M3 ? 2 : 1];
  __device__ __forceinline__ explicit Frag(const uint4& u) {
    if constexpr (TYPE == T_E4M3) {
      v[0] = __builtin_bit_cast(uint4, e4m3_half(u, 0));
      v[1] = __builtin_bit_cast(uint4, e4m3_half(u, 1));
    } else {
      v[0] = u;
    }
  }
};
template <int TYPE>
__device__ __forceinline__ void mma(const Frag<TYPE>& w, const Frag<TYPE>& x, typename Mma<TYPE>::Acc& acc) {
  if constexpr (TYPE == T_E4M3) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_h8(w.v[0]), as_h8(x.v[0]), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_h8(w.v[1]), as_h8(x.v[1]), acc, 0, 0, 0);
  } else if constexpr (TYPE == T_INT8) {
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(as_i4(w.v[0]), as_i4(x.v[0]), acc, 0, 0, 0);
  } else if constexpr (TYPE == T_F16) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_h8(w.v[0]), as_h8(x.v[0]), acc, 0, 0, 0);
  } else {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf8(w.v[0]), as_bf8(x.v[0]), acc, 0, 0, 0);
  }
}

// Waits for the wave's LDS reads and all but its N most recent vector-memory operations.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
  asm volatile("" ::: "memory");
}

template <int TYPE, int TI>
__global__ void __launch_bounds__(256) k_gemm_few(Args a) {
  constexpr int R = TI == 1 ? 3 : 2;
  constexpr int L = 2 + 2 * TI;              // LDS-DMA instructions (8 rows each) of a stage
  constexpr int BUF = 1024 * L;              // of one wave
  using Acc = typename Mma<TYPE>::Acc;
  __shared__ __attribute__((aligned(16))) uint8_t b0[4 * BUF];
  __shared__ __attribute__((aligned(16))) uint8_t b1[4 * BUF];
  __shared__ __attribute__((aligned(16))) uint8_t b2[R > 2 ? 4 * BUF : 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int q = lane >> 4, r16 = lane & 15;
  const int n0 = blockIdx.x * 16, nrows = min(16, a.N - n0);
  const rsrc_t rw = make_rsrc(a.w + (int64_t)n0 * a.KB, (size_t)nrows * a.KB);
  const rsrc_t rx = make_rsrc(a.x, (size_t)((a.M - 1) * a.x_stride + a.KB));
  // instruction i moves rows 8 i ... 8 i + 7: lane l slot l % 8 of row 8 i + l / 8
  uint32_t vo[L];
#pragma unroll
  for (int i = 0; i < L; i++) {
    const int row = (i < 2 ? i : i - 2) * 8 + (lane >> 3);
    const int piece = (lane & 7) ^ ((row >> 1) & 7);
    vo[i] = i < 2 ? (row < nrows ? (uint32_t)row * (uint32_t)a.KB + 16u * piece : kPast)
                  : (row < a.M ? (uint32_t)row * (uint32_t)a.x_stride + 16u * piece : kPast);
  }
  // pieces of rows 8 i + l / 8 for even and odd i
  const int pe = 16 * ((lane & 7) ^ (lane >> 4)), po = 16 * ((lane & 7) ^ (4 + (lane >> 4)));
  auto load = [&](int st, uint8_t* b) {      // stage st of this wave; pieces past the end of K read as zeros
    const int k0 = (st * 4 + wave) * BK;
    const bool e = k0 + pe >= a.KB, o = k0 + po >= a.KB;
#pragma unroll
    for (int i = 0; i < L; i++)
      dma16(i < 2 ? rw : rx, b + wave * BUF + i * 1024, (i & 1 ? o : e) ? kPast : vo[i], (uint32_t)k0);
  };
  Acc acc[TI];
#pragma unroll
  for (int t = 0; t < TI; t++)
#pragma unroll
    for (int i = 0; i < 4; i++) acc[t][i] = 0;
  const int chunks = (a.KB + BK - 1) / BK;
  const int stages = (chunks + 3) / 4;       // the last may be past the end for some waves: zeros
  auto step = [&](int st, uint8_t* b) {
    wait_loads<(R - 1) * L>();               // stage st is in
    uint4 w[2], x[TI][2];
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const int at = wave * BUF + r16 * BK + 16 * ((q + 4 * j) ^ ((r16 >> 1) & 7));
      w[j] = lds_piece(b, at);
#pragma unroll
      for (int t = 0; t < TI; t++) x[t][j] = lds_piece(b, at + 2048 + t * 16 * BK);
    }
    wait_loads<(R - 1) * L>();               // the reads are done: the stage's bytes may be loaded again
    load(st + R, b);
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const Frag<TYPE> fw(w[j]);
#pragma unroll
      for (int t = 0; t < TI; t++) mma<TYPE>(fw, Frag<TYPE>(x[t][j]), acc[t]);
    }
  };
  load(0, b0);
  load(1, b1);
  if (R > 2) load(2, b2);
  // the epilogue's operands: thread t < 64 TI ends up with columns n ... n + 3 of row m
  const int ot = threadIdx.x >> 6, m = ot * 16 + r16, n = n0 + 4 * q;
  const bool mine = ot < TI && m < a.M;
  float sx = 1.f, sw[4], bv[4];
  uint32_t rr[2] = {0, 0};
  if (mine && a.xs) sx = a.xs[m];
  if (mine && a.res && n < a.N) load_piece<4>(a.res, m * a.res_stride + n, a.N - n, rr);
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const bool in = mine && n + j < a.N;
    sw[j] = in && a.ws ? a.ws[n + j] : 1.f;
    bv[j] = in && a.bias ? load16(a.bias, n + j, a.bf) : 0.f;
  }
  for (int st = 0; st < stages; st += R) {   // stages past the last are zeros
    step(st, b0);
    step(st + 1, b1);
    if (R > 2) step(st + 2, b2);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");     // nothing of the rings may land in the partial sums
  __syncthreads();
  Acc* red = reinterpret_cast<Acc*>(b0);     // [4 waves][TI][64 lanes]
#pragma unroll
  for (int t = 0; t < TI; t++) red[(wave * TI + t) * 64 + lane] = acc[t];
  __syncthreads();
  if (!mine) return;
  Acc v = red[ot * 64 + lane];
#pragma unroll
  for (int w = 1; w < 4; w++) v += red[(w * TI + ot) * 64 + lane];
  float y[4], rv[4];
  unpack4(rr, a.bf, rv);
#pragma unroll
  for (int j = 0; j < 4; j++) y[j] = activate((float)v[j] * sx * sw[j] + bv[j], a.act) + rv[j];
  const uint32_t o[2] = {pack16(y[0], y[1], a.bf), pack16(y[2], y[3], a.bf)};
  if (n < a.N) store_piece<4>(a.y, m * a.y_stride + n, a.N - n, o);
}

template <int TYPE>
hipError_t launch_type(const Args& a, hipStream_t s) {
  const dim3 grid((a.N + 15) / 16), block(256);
  switch ((a.M + 15) / 16) {
    case 1: hipLaunchKernelGGL((k_gemm_few<TYPE, 1>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((k_gemm_few<TYPE, 2>), grid, block, 0, s, a); break;
    case 3: hipLaunchKernelGGL((k_gemm_few<TYPE, 3>), grid, block, 0, s, a); break;
    case 4: hipLaunchKernelGGL((k_gemm_few<TYPE, 4>), grid, block, 0, s, a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_few(const Args& a, int type, hipStream_t s) {
  switch (type) {
    case T_INT8: return launch_type<T_INT8>(a, s);
    case T_E4M3: return launch_type<T_E4M3>(a, s);
    case T_F16: return launch_type<T_F16>(a, s);
    case T_BF16: return launch_type<T_BF16>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace gact
}  // namespace svdq
