// C-ABI layer of the operators between the quantized linears (include/svdq.h): host-side
// argument validation and kernel launches.  Every check happens before any HIP call; no
// exception leaves this file.
#include <math.h>

#include "../../include/svdq.h"
#include "block_ops.h"

using namespace svdq;

namespace {

constexpr int kMaxDim = 1 << 24;
constexpr int64_t kMaxStride = (int64_t)1 << 40;     // elements: keeps every index product below 2^63
constexpr int64_t kMaxRowBytes = (int64_t)4 << 20;   // 256 rows are addressed with 31-bit byte offsets

inline bool is16(int t) { return t == SVDQ_TYPE_F16 || t == SVDQ_TYPE_BF16; }
inline bool is8(int t) { return t == SVDQ_TYPE_INT8 || t == SVDQ_TYPE_E4M3; }
inline int bytes_of(int t) { return is8(t) ? 1 : is16(t) ? 2 : 4; }
inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool stride_ok(int64_t s, int64_t least) { return s >= least && s <= kMaxStride; }
inline bool eps_ok(float e) { return isfinite(e) && e > 0.f; }

svdq_status check_product(int M, int N, int K, int type) {
  if (M < 0 || N < 0 || K <= 0 || M > kMaxDim || N > kMaxDim || (int64_t)K * bytes_of(type) > kMaxRowBytes)
    return SVDQ_ERR_SHAPE;
  if (K * bytes_of(type) % 16 != 0 || (type == SVDQ_TYPE_INT8 && K > 1 << 17)) return SVDQ_ERR_SHAPE;
  if (((int64_t)M + 63) / 64 * (((int64_t)N + 63) / 64) >= (int64_t)1 << 31) return SVDQ_ERR_SHAPE;
  return SVDQ_OK;
}

svdq_status map_launch(hipError_t e) {
  if (e == hipSuccess) return SVDQ_OK;
  if (e == hipErrorInvalidConfiguration) return SVDQ_ERR_SHAPE;   // !launchable
  if (e == hipErrorNoBinaryForGpu || e == hipErrorInvalidDeviceFunction) return SVDQ_ERR_DEVICE;
  return SVDQ_ERR_LAUNCH;
}

}  // namespace

extern "C" {

svdq_status svdq_add_rmsnorm(const void* x, int64_t x_stride, svdq_type x_type, const void* residual,
                             int64_t residual_stride, svdq_type residual_type, const void* weight,
                             svdq_type weight_type, float eps, int M, int K, svdq_type out_type, void* out,
                             float* scales, void* residual_out, int64_t residual_out_stride, void* stream) {
  if (!is16(x_type) || (weight_type != x_type && weight_type != SVDQ_TYPE_F32) ||
      (out_type != x_type && !is8(out_type)))
    return SVDQ_ERR_FORMAT;
  if (residual && residual_type != x_type && residual_type != SVDQ_TYPE_F32) return SVDQ_ERR_FORMAT;
  if (M < 0 || M > kMaxDim || K <= 0 || K > kMaxDim || !eps_ok(eps)) return SVDQ_ERR_SHAPE;
  if (!stride_ok(x_stride, K)) return SVDQ_ERR_SHAPE;
  if (residual && (!stride_ok(residual_stride, K) || !stride_ok(residual_out_stride, K))) return SVDQ_ERR_SHAPE;
  if (M == 0) return SVDQ_OK;
  if (!x || !weight || !out || (is8(out_type) && !scales) || (residual && !residual_out)) return SVDQ_ERR_NULL;
  if (!aligned(x, 2) || !aligned(weight, bytes_of(weight_type)) || !aligned(out, bytes_of(out_type)) ||
      !aligned(scales, 4))
    return SVDQ_ERR_ALIGN;
  if (residual && (!aligned(residual, bytes_of(residual_type)) || !aligned(residual_out, bytes_of(residual_type))))
    return SVDQ_ERR_ALIGN;
  const NormArgs a{x, x_stride, x_type, residual, residual_stride, residual_type, weight, weight_type,
                   eps, M, K, out_type, out, scales, residual_out, residual_out_stride};
  return map_launch(launch_rmsnorm(a, static_cast<hipStream_t>(stream)));
}

svdq_status svdq_gemm_act_residual(const void* x, int64_t x_stride, const float* xs, const void* w,
                                   const float* ws, const void* bias, const void* residual,
                                   int64_t residual_stride, int M, int N, int K, svdq_type type,
                                   svdq_activation act, svdq_type out_type, void* y, int64_t y_stride,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  if ((!is8(type) && !is16(type)) || !is16(out_type)) return SVDQ_ERR_FORMAT;
  if (act != SVDQ_ACT_NONE && act != SVDQ_ACT_GELU_TANH && act != SVDQ_ACT_SILU) return SVDQ_ERR_FORMAT;
  const int b = bytes_of(type);
  const svdq_status st = check_product(M, N, K, type);
  if (st != SVDQ_OK) return st;
  if (x_stride < K || x_stride > kMaxRowBytes / b || x_stride * b % 16 != 0) return SVDQ_ERR_SHAPE;
  if (!stride_ok(y_stride, N) || (residual && !stride_ok(residual_stride, N))) return SVDQ_ERR_SHAPE;
  if (M == 0 || N == 0) return SVDQ_OK;
  if (!x || !w || !y) return SVDQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 2) || !aligned(xs, 4) || !aligned(ws, 4) ||
      !aligned(bias, 2) || !aligned(residual, 2) || !aligned(workspace, 16))
    return SVDQ_ERR_ALIGN;
  const GemmActArgs a{x, x_stride, xs, w, ws, bias, residual, residual_stride, M, N, K, type, act, out_type, y, y_stride,
                      workspace, workspace ? workspace_bytes : 0};
  return map_launch(launch_gemm_act(a, static_cast<hipStream_t>(stream)));
}

size_t svdq_gemm_act_residual_workspace_bytes(int M, int N, int K, svdq_type type) {
  if ((!is8(type) && !is16(type)) || check_product(M, N, K, type) != SVDQ_OK || M == 0 || N == 0) return 0;
  return gemm_act_plan(M, N, K, type, ~(size_t)0).bytes;
}

const char* svdq_gemm_act_residual_kernel(int M, int N, int K, svdq_type type, size_t workspace_bytes, int* splits,
                                          int* tail) {
  if ((!is8(type) && !is16(type)) || check_product(M, N, K, type) != SVDQ_OK || M == 0 || N == 0) return nullptr;
  const GemmActPlan p = gemm_act_plan(M, N, K, type, workspace_bytes);
  if (splits) *splits = p.splits;
  if (tail) *tail = p.tail;
  switch (p.kind) {
    case GemmActPlan::FEW: return "few rows";
    case GemmActPlan::T64: return "64x64";
    case GemmActPlan::T64x128: return "64x128";
    case GemmActPlan::T128x192: return "128x192";
    case GemmActPlan::T128x256: return "128x256";
    default: return "256x256";
  }
}

svdq_status svdq_rope_axes(const svdq_rope_operand* operands, int count, int batch, int tokens, int dim,
                           svdq_type type, const void* positions, int positions_fp32, int64_t position_batch,
                           const float* inv_freq, int axes, const int* axis_pairs, int halves, float eps,
                           int inverse, void* stream) {
  if (!is16(type)) return SVDQ_ERR_FORMAT;
  if (!operands || !axis_pairs) return SVDQ_ERR_NULL;
  if (count < 1 || count > 2 || batch < 0 || tokens < 0 || batch > kMaxDim || tokens > kMaxDim) return SVDQ_ERR_SHAPE;
  if (dim < 1 || dim > 1024 || axes < 1 || axes > kMaxRopeAxes || !stride_ok(position_batch, 0)) return SVDQ_ERR_SHAPE;
  RopeArgs a{};
  for (int i = 0; i < axes; i++) {
    if (axis_pairs[i] < 0 || axis_pairs[i] > dim) return SVDQ_ERR_SHAPE;
    a.pairs += axis_pairs[i];
    a.end[i] = a.pairs;
  }
  for (int i = axes; i < kMaxRopeAxes; i++) a.end[i] = a.pairs;
  if (a.pairs < 1 || 2 * a.pairs > dim) return SVDQ_ERR_SHAPE;
  int64_t heads = 0;
  for (int i = 0; i < count; i++) {
    const svdq_rope_operand& o = operands[i];
    if (o.heads < 1 || o.heads > kMaxDim) return SVDQ_ERR_SHAPE;
    for (const int64_t s : {o.in_batch, o.in_token, o.in_head, o.out_batch, o.out_token, o.out_head})
      if (!stride_ok(s, 0)) return SVDQ_ERR_SHAPE;
    if (o.weight && inverse) return SVDQ_ERR_FORMAT;
    if (o.weight && !eps_ok(eps)) return SVDQ_ERR_SHAPE;
    heads += o.heads;
  }
  // one workgroup takes at least one head of one token
  if ((int64_t)batch * tokens > (int64_t)1 << 30 || (int64_t)batch * tokens * heads >= (int64_t)1 << 31)
    return SVDQ_ERR_SHAPE;
  if (batch == 0 || tokens == 0) return SVDQ_OK;
  if (!positions || !inv_freq) return SVDQ_ERR_NULL;
  if (!aligned(positions, 4) || !aligned(inv_freq, 4)) return SVDQ_ERR_ALIGN;
  for (int i = 0; i < count; i++) {
    const svdq_rope_operand& o = operands[i];
    if (!o.in || !o.out) return SVDQ_ERR_NULL;
    if (!aligned(o.in, 2) || !aligned(o.out, 2) || !aligned(o.weight, 4)) return SVDQ_ERR_ALIGN;
    a.op[i] = RopeOperand{o.in, o.out, o.weight, o.heads, o.in_batch, o.in_token, o.in_head,
                          o.out_batch, o.out_token, o.out_head};
  }
  a.nops = count;
  a.batch = batch;
  a.tokens = tokens;
  a.dim = dim;
  a.type = type;
  a.positions = positions;
  a.pos_batch = position_batch;
  a.pos_token = axes;
  a.pos_float = positions_fp32 != 0;
  a.inv_freq = inv_freq;
  a.axes = axes;
  a.halves = halves != 0;
  a.inverse = inverse != 0;
  a.eps = eps;
  return map_launch(launch_rope(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
