// Host-side argument validation of the block operators' C ABI (include/svdq.h), exercised without
// a GPU in a build of the library's host code with AddressSanitizer and
// UndefinedBehaviorSanitizer.  Every call returns before any HIP call; pointers are fake.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>

#include "../include/svdq.h"

namespace {
int failures = 0;
void expect(const char* what, int got, int want) {
  if (got != want) {
    std::printf("FAIL %s: status %d, expected %d\n", what, got, want);
    failures++;
  }
}
void* const P = reinterpret_cast<void*>(4096);
float* const PF = reinterpret_cast<float*>(4096);
const svdq_type BAD = static_cast<svdq_type>(123456789);
const int64_t HUGE64 = std::numeric_limits<int64_t>::max(), LOW64 = std::numeric_limits<int64_t>::min();
const int HUGE32 = std::numeric_limits<int>::max(), LOW32 = std::numeric_limits<int>::min();
}  // namespace

int main() {
  const svdq_type H = SVDQ_TYPE_F16, F = SVDQ_TYPE_F32, I = SVDQ_TYPE_INT8;
  auto norm = [&](int64_t xs, svdq_type xt, float eps, int M, int K, svdq_type ot) {
    return svdq_add_rmsnorm(P, xs, xt, P, xs, F, P, F, eps, M, K, ot, P, PF, P, xs, nullptr);
  };
  expect("norm type", norm(64, BAD, 1e-6f, 4, 64, I), SVDQ_ERR_FORMAT);
  expect("norm out type", norm(64, H, 1e-6f, 4, 64, BAD), SVDQ_ERR_FORMAT);
  expect("norm stride", norm(HUGE64, H, 1e-6f, 4, 64, I), SVDQ_ERR_SHAPE);
  expect("norm negative stride", norm(LOW64, H, 1e-6f, 4, 64, I), SVDQ_ERR_SHAPE);
  expect("norm rows", norm(64, H, 1e-6f, HUGE32, 64, I), SVDQ_ERR_SHAPE);
  expect("norm columns", norm(64, H, 1e-6f, 4, LOW32, I), SVDQ_ERR_SHAPE);
  expect("norm eps", norm(64, H, NAN, 4, 64, I), SVDQ_ERR_SHAPE);
  expect("norm empty", norm(64, H, 1e-6f, 0, 64, I), SVDQ_OK);
  auto gemm = [&](int64_t xs, int M, int N, int K, svdq_type t, svdq_activation act, int64_t ys) {
    return svdq_gemm_act_residual(P, xs, PF, P, PF, P, P, ys, M, N, K, t, act, H, P, ys, P, 0, nullptr);
  };
  expect("gemm type", gemm(64, 4, 32, 64, BAD, SVDQ_ACT_NONE, 32), SVDQ_ERR_FORMAT);
  expect("gemm act", gemm(64, 4, 32, 64, I, static_cast<svdq_activation>(LOW32), 32), SVDQ_ERR_FORMAT);
  expect("gemm K", gemm(64, 4, 32, HUGE32, H, SVDQ_ACT_NONE, 32), SVDQ_ERR_SHAPE);
  expect("gemm stride", gemm(HUGE64, 4, 32, 64, H, SVDQ_ACT_NONE, 32), SVDQ_ERR_SHAPE);
  expect("gemm y stride", gemm(64, 4, 32, 64, H, SVDQ_ACT_NONE, HUGE64), SVDQ_ERR_SHAPE);
  expect("gemm rows", gemm(64, LOW32, 32, 64, H, SVDQ_ACT_NONE, 32), SVDQ_ERR_SHAPE);
  expect("gemm empty", gemm(64, 0, 32, 64, H, SVDQ_ACT_NONE, 32), SVDQ_OK);
  svdq_rope_operand op[2] = {{P, P, nullptr, 2, 512, 128, 64, 512, 128, 64}, {P, P, nullptr, 2, 512, 128, 64, 512, 128, 64}};
  int pairs[SVDQ_ROPE_MAX_AXES] = {8, 24, 0, 0};
  auto rope = [&](int B, int T, int D, int axes, svdq_type t) {
    return svdq_rope_axes(op, 2, B, T, D, t, P, 0, 0, PF, axes, pairs, 0, 1e-6f, 0, nullptr);
  };
  expect("rope type", rope(1, 4, 64, 2, BAD), SVDQ_ERR_FORMAT);
  expect("rope axes", rope(1, 4, 64, HUGE32, H), SVDQ_ERR_SHAPE);
  expect("rope dim", rope(1, 4, LOW32, 2, H), SVDQ_ERR_SHAPE);
  expect("rope size", rope(1 << 24, 1 << 24, 64, 2, H), SVDQ_ERR_SHAPE);
  op[1].heads = HUGE32;
  expect("rope heads", rope(1, 4, 64, 2, H), SVDQ_ERR_SHAPE);
  op[1].heads = 1 << 24;
  expect("rope units", rope(1 << 10, 1 << 20, 64, 2, H), SVDQ_ERR_SHAPE);
  op[1].heads = 2;
  op[0].in_token = LOW64;
  expect("rope stride", rope(1, 4, 64, 2, H), SVDQ_ERR_SHAPE);
  op[0].in_token = 128;
  pairs[0] = pairs[1] = HUGE32;
  expect("rope pairs", rope(1, 4, 64, 2, H), SVDQ_ERR_SHAPE);
  pairs[0] = 8;
  pairs[1] = 24;
  expect("rope empty", rope(1, 0, 64, 2, H), SVDQ_OK);
  std::printf("%s: %d failure(s)\n", failures ? "FAILED" : "OK", failures);
  return failures ? 1 : 0;
}
