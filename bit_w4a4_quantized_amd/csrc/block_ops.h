// Shared pieces of the operators between the quantized linears (k_rmsnorm.hip, k_rope.hip,
// k_gemm_act.hip): element types, their conversions, and the argument structs block_api.hip
// fills.  Arithmetic is fp32; every conversion to a narrower type rounds to nearest even.
#pragma once
#include "kernels.h"

namespace svdq {

enum Type { T_F16 = 0, T_BF16 = 1, T_F32 = 2, T_INT8 = 3, T_E4M3 = 4 };
enum Act { ACT_NONE = 0, ACT_GELU = 1, ACT_SILU = 2 };

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf16_f32(uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ float f16_f32(uint32_t bits) { return __half2float(__ushort_as_half((unsigned short)bits)); }

// A 16-bit value of either type; `bf` is uniform.
__device__ __forceinline__ float load16(const void* p, int64_t i, bool bf) {
  const uint32_t b = static_cast<const uint16_t*>(p)[i];
  return bf ? bf16_f32(b) : f16_f32(b);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), f16x2));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
__device__ __forceinline__ uint32_t pack16(float a, float b, bool bf) { return bf ? pack_bf16(a, b) : pack_f16(a, b); }
__device__ __forceinline__ void store16(void* p, int64_t i, float v, bool bf) {
  static_cast<uint16_t*>(p)[i] = (uint16_t)pack16(v, v, bf);
}
__device__ __forceinline__ float round16(float v, bool bf) {
  const uint32_t b = pack16(v, v, bf) & 0xFFFFu;
  return bf ? bf16_f32(b) : f16_f32(b);
}

// Eight 16-bit values of a 16-byte piece, to and from fp32.
__device__ __forceinline__ void unpack8(const uint4& u, bool bf, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if (bf) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      f[2 * i] = bf16_f32(w[i] & 0xFFFFu);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      f[2 * i] = f16_f32(w[i] & 0xFFFFu);
      f[2 * i + 1] = f16_f32(w[i] >> 16);
    }
  }
}
__device__ __forceinline__ uint4 pack8(const float* f, bool bf) {
  uint4 u;
  if (bf) {
    u = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  } else {
    u = make_uint4(pack_f16(f[0], f[1]), pack_f16(f[2], f[3]), pack_f16(f[4], f[5]), pack_f16(f[6], f[7]));
  }
  return u;
}

// A launch holds fewer than 2^32 threads.
inline bool launchable(int64_t blocks, int threads) { return blocks * threads < (int64_t)1 << 32; }

struct NormArgs {
  const void* x; int64_t x_stride; int x_type;                  // strides in elements
  const void* res; int64_t res_stride; int res_type;            // res may be null
  const void* weight; int weight_type;
  float eps; int M, K; int out_type;
  void* out; float* scales; void* res_out; int64_t res_out_stride;
};
hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t s);

struct RopeOperand {
  const void* in; void* out; const float* weight; int heads;
  int64_t in_batch, in_token, in_head, out_batch, out_token, out_head;   // strides in elements
};
constexpr int kMaxRopeAxes = 4;
struct RopeArgs {
  RopeOperand op[2]; int nops;
  int batch, tokens, dim, type;
  const void* positions; int64_t pos_batch, pos_token; int pos_float;
  const float* inv_freq;
  int axes, pairs, end[kMaxRopeAxes];        // pairs before end[a] (and not before end[a - 1]) turn by axis a
  int halves, inverse; float eps;
};
hipError_t launch_rope(const RopeArgs& a, hipStream_t s);

struct GemmActArgs {
  const void* x; int64_t x_stride; const float* xs; const void* w; const float* ws;
  const void* bias; const void* res; int64_t res_stride;
  int M, N, K, type, act, out_type;
  void* y; int64_t y_stride;
  void* part; size_t part_bytes;             // room for the sums of K's splits (may be null)
};
// The kernel a product takes, and the bytes its splits of K need (0: one split); with less room than
// `part_bytes` K is split less or not at all.  LARGE: the tiles taken as they are, and the parts that
// each of the others, a last partial round, is cut into (0: there are none).
struct GemmActPlan {
  enum Kind { FEW, T64, T64x128, T128x192, T128x256, LARGE };
  int kind, splits;
  size_t bytes;
  int whole, tail;
};
GemmActPlan gemm_act_plan(int M, int N, int K, int type, size_t part_bytes);
hipError_t launch_gemm_act(const GemmActArgs& a, hipStream_t s);

}  // namespace svdq
