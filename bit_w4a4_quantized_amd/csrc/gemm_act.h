// Shared by the kernels of svdq_gemm_act_residual (k_gemm_act.hip, k_gemm_few.hip):
//
//   y[m, n] = rnd( act( (sum_k x[m, k] w[n, k]) xs[m] ws[n] + b[n] ) + res[m, n] )
//
// for int8 (exact int32 sums), FP8 E4M3, fp16 and bf16 operands (fp32 sums), both row-major
// with K contiguous.  The kernels see rows of bytes: a lane's MFMA operands come from one 16-byte
// piece of its row, whatever the type, so staging and layout are the same for all four.
//
// E4M3 operands become fp16 in registers, exactly, and go through the fp16 matrix instructions, at
// half the FP8 rate.  The FP8 instructions add eight products at a time, aligned to the largest of
// the eight with 13 bits below it (in both of their forms), so that small products beside a large
// one are lost: of the whole-number sums of test_gemm_sums_beside_large_products, all below 2048,
// they miss almost every one, by up to 83.  They would take 15.1 us at 64 x 12288 x 3072 (16.0 in
// fp16) and 162 at 4608 x 3072 x 12288 (268; bf16 operands 312).
#pragma once
#include "block_ops.h"
#include "gemm_skel.h"

namespace svdq {
namespace gact {

using skel::dma16;

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int BK = 128;                      // bytes of K a stage: a whole cache line of each row
constexpr uint32_t kPast = 0x80000000u;      // an offset past every resource's range: loads give zeros

// What the kernels take, with strides and K in bytes.
struct Args {
  const uint8_t* x; int64_t x_stride; const float* xs; const uint8_t* w; const float* ws;
  const void* bias; const void* res; int64_t res_stride;
  int M, N, KB, act, bf;                     // bf: 16-bit output is bf16
  void* y; int64_t y_stride;
};

__device__ __forceinline__ v8bf as_bf8(const uint4& u) { return __builtin_bit_cast(v8bf, u); }
// The piece at byte `at` of a ring buffer, in one access one step away from the buffer's name: the
// compiler then knows which buffer it reads, and does not wait for the loads into the others.
__device__ __forceinline__ uint4 lds_piece(const uint8_t* buf, int at) {
  return as_u4(*reinterpret_cast<const u32x4_t*>(buf + at));
}

// The sixteen E4M3 codes of a piece as fp16, the first eight and the rest.
__device__ __forceinline__ v8h e4m3_half(const uint4& u, int half) {
  const uint32_t a = half ? u.z : u.x, b = half ? u.w : u.y;
  const f16x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false), __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true),
                      __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false), __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true)};
  return __builtin_bit_cast(v8h, v);
}

__device__ __forceinline__ float activate(float v, int act) {
  if (act == ACT_GELU) return gelu_div(v, 1.0f);
  if (act == ACT_SILU) return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * v));
  return v;
}

// The first min(n, E) of E (4 or 8) 16-bit values at base + at, which has any alignment, zeros
// behind them; and back.  Global accesses need no more than the elements' alignment, so an odd
// row stride costs no narrow accesses (f16 333 x 1048 x 1999: 10.8 us, 14.6 with one element at
// a time where the rows are not 16-byte aligned).
template <int E>
__device__ __forceinline__ void load_piece(const void* base, int64_t at, int n, uint32_t (&v)[E / 2]) {
  const uint16_t* p = static_cast<const uint16_t*>(base) + at;
  if (n >= E) {
    __builtin_memcpy(v, p, 2 * E);
  } else {
#pragma unroll
    for (int i = 0; i < E / 2; i++)
      v[i] = (2 * i < n ? p[2 * i] : 0u) | ((2 * i + 1 < n ? p[2 * i + 1] : 0u) << 16);
  }
}
template <int E>
__device__ __forceinline__ void store_piece(void* base, int64_t at, int n, const uint32_t (&v)[E / 2]) {
  uint16_t* p = static_cast<uint16_t*>(base) + at;
  if (n >= E) {
    __builtin_memcpy(p, v, 2 * E);
  } else {
#pragma unroll
    for (int i = 0; i < E - 1; i++)
      if (i < n) p[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
  }
}
// Four values of a piece in fp32, and four rounded.
__device__ __forceinline__ void unpack4(const uint32_t (&v)[2], bool bf, float* f) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t b = (v[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
    f[i] = bf ? bf16_f32(b) : f16_f32(b);
  }
}

hipError_t launch_few(const Args& a, int type, hipStream_t s);
constexpr int kFewRows = 64;                 // rows launch_few takes

}  // namespace gact
}  // namespace svdq
