// Host-side argument validation of the operators around a paged cache (include/svdq.h), and the lookups
// that their kernels make in tables and starts that the host never sees, exercised without a GPU in a
// build of the library's host code with AddressSanitizer and UndefinedBehaviorSanitizer.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>
#include <vector>

#include "../bit_w4a4_quantized_amd/csrc/slots.h"
#include "../include/svdq.h"

namespace {
int failures = 0;
void expect(const char* what, long long got, long long want) {
  if (got != want) {
    std::printf("FAIL %s: %lld, expected %lld\n", what, got, want);
    failures++;
  }
}
void* const P = reinterpret_cast<void*>(4096);
float* const PF = reinterpret_cast<float*>(4096);
int* const PI = reinterpret_cast<int*>(4096);
const svdq_type BAD = static_cast<svdq_type>(123456789);
const int64_t HUGE64 = std::numeric_limits<int64_t>::max(), LOW64 = std::numeric_limits<int64_t>::min();
const int HUGE32 = std::numeric_limits<int>::max(), LOW32 = std::numeric_limits<int>::min();
}  // namespace

int main() {
  svdq_paged_cache c{P, P, PF, PF, SVDQ_TYPE_INT8, 9, 16, 2, 64, 2048, 128, 64, 32, 2, 1};
  svdq_paged_batch b{PI, 4, 4, PI, PI, 3};
  svdq_rope_operand q{P, P, nullptr, 4, 0, 256, 64, 0, 256, 64}, k{P, nullptr, nullptr, 2, 0, 128, 64, 0, 0, 0};
  int pairs[SVDQ_ROPE_MAX_AXES] = {8, 24, 0, 0};
  const svdq_type H = SVDQ_TYPE_F16;
  auto append = [&](int tokens, int axes, svdq_type t) {
    return svdq_rope_append(&c, &b, &q, &k, P, 128, 64, tokens, t, P, 0, PF, axes, pairs, 0, 1e-6f, nullptr);
  };
  auto attention = [&](int heads, int tokens, int64_t stride, float scale) {
    return svdq_tree_attention(&c, &b, P, stride, 64, heads, tokens, H, scale, P, stride, 8, P, stride, 64, P, 0, nullptr);
  };
  auto keep = [&](int64_t stride, int width) { return svdq_cache_keep(&c, &b, PI, stride, width, nullptr); };
  expect("append type", append(4, 2, BAD), SVDQ_ERR_FORMAT);
  expect("append tokens", append(HUGE32, 2, H), SVDQ_ERR_SHAPE);
  expect("append axes", append(4, LOW32, H), SVDQ_ERR_SHAPE);
  pairs[0] = pairs[1] = HUGE32;
  expect("append pairs", append(4, 2, H), SVDQ_ERR_SHAPE);
  pairs[0] = 8;
  pairs[1] = 24;
  expect("append empty", append(0, 2, H), SVDQ_OK);
  expect("attention heads", attention(HUGE32, 4, 256, 1.f), SVDQ_ERR_SHAPE);
  expect("attention tokens", attention(4, LOW32, 256, 1.f), SVDQ_ERR_SHAPE);
  expect("attention stride", attention(4, 4, HUGE64, 1.f), SVDQ_ERR_SHAPE);
  expect("attention scale", attention(4, 4, 256, NAN), SVDQ_ERR_SHAPE);
  expect("attention empty", attention(4, 0, 256, 1.f), SVDQ_OK);
  expect("keep stride", keep(LOW64, 4), SVDQ_ERR_SHAPE);
  expect("keep width", keep(4, HUGE32), SVDQ_ERR_SHAPE);
  expect("keep empty", keep(4, 0), SVDQ_OK);
  for (const int64_t s : {HUGE64, LOW64, (int64_t)-64}) {
    const svdq_paged_cache saved = c;
    c.page_stride = s;
    expect("page stride", keep(4, 4), SVDQ_ERR_SHAPE);
    c = saved;
    c.scale_token_stride = s;
    expect("scale stride", keep(4, 4), SVDQ_ERR_SHAPE);
    c = saved;
    c.pages = s;
    expect("pages", keep(4, 4), SVDQ_ERR_SHAPE);
    c = saved;
  }
  for (const int n : {HUGE32, LOW32, 0, 48}) {
    const svdq_paged_cache saved = c;
    c.page_size = n;
    expect("page size", keep(4, 4), SVDQ_ERR_SHAPE);
    c = saved;
    c.dim = n == 48 ? 40 : n;
    expect("dim", keep(4, 4), SVDQ_ERR_SHAPE);
    c = saved;
  }
  b.table_width = HUGE32;
  expect("table width", keep(4, 4), SVDQ_ERR_SHAPE);
  expect("workspace", (long long)svdq_tree_attention_workspace_bytes(HUGE32, HUGE32, HUGE32, 1, 128, HUGE32, HUGE32), 0);

  // tables, starts and contexts with anything in them: no read outside, no page outside
  using namespace svdq;
  const int pages = 7, width = 3, shift = 2;
  const std::vector<int> table = {0, 6, 7, -1, LOW32, HUGE32, 3, 2, 1};
  const std::vector<int> starts = {-5, LOW32, HUGE32, 4}, context = {HUGE32, LOW32, 3};
  PagedCache pc{};
  pc.pages = pages;
  pc.shift = shift;
  PagedBatch pb{table.data(), width, width, starts.data(), context.data(), 3};
  for (int s = 0; s < 3; s++) {
    for (const int slot : {0, 3, 4, 7, 8, 11, 12, 13, 1 << 30, HUGE32}) {
      const int col = slot >> shift, want = col < width && (unsigned)table[s * width + col] < 7u ? table[s * width + col] : -1;
      expect("page", page_of(pb, pc, s, slot), want);
    }
    const int ctx = context_of(pb, s);
    expect("context", ctx, s == 0 ? 1 << 30 : s == 1 ? 0 : 3);
  }
  for (int i = 0; i < 4; i++) {
    const int at = start_of(pb, i, 10);
    expect("start", at, i == 2 ? 10 : i == 3 ? 4 : 0);
  }
  std::printf("%s: %d failure(s)\n", failures ? "FAILED" : "OK", failures);
  return failures ? 1 : 0;
}
