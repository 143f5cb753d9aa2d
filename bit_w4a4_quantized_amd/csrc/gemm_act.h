// Shared by the kernels of svdq_gemm_act_residual (k_gemm_act.hip, k_gemm_few.hip):
//
//   y[m, n] = rnd( act( (sum_k x[m, k] w[n, k]) xs[m] ws[n] + b[n] ) + res[m, n] )
//
// for int8 (exact int32 sums), FP8 E4M3, fp16 and bf16 operands (fp32 sums), both row-major
// with K contiguous.  The kernels see rows of bytes: a lane's MFMA operand is one 16-byte piece
// of its row (two for FP8), whatever the type, so staging and layout are the same for all four.
//
// FP8: the matrix core adds eight products at a time, aligned to the largest of the eight with 13
// bits below it (found with one large and several small products; the FP8 instructions of half
// the rate do the same), and the eights' sums in fp32.  The codes themselves carry 3 bits, so the
// lost bits are far below theirs; converting to fp16 first would keep them at half the rate.
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
  int wide;                                  // elements of y and res that may be moved at once: 8, 4 or 1
  void* y; int64_t y_stride;
};

__device__ __forceinline__ v8bf as_bf8(const uint4& u) { return __builtin_bit_cast(v8bf, u); }
__device__ __forceinline__ v8i as_i8(const uint4& a, const uint4& b) {
  return v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

__device__ __forceinline__ float activate(float v, int act) {
  if (act == ACT_GELU) return gelu_div(v, 1.0f);
  if (act == ACT_SILU) return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * v));
  return v;
}

hipError_t launch_few(const Args& a, int type, hipStream_t s);
constexpr int kFewRows = 64;                 // rows launch_few takes

}  // namespace gact
}  // namespace svdq
