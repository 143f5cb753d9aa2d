// Which rows of attention a slot takes, for starts that hold anything: whatever sequence is found for a slot, its rows are
// tokens and heads that there are.  And the quotients that the kernels take without dividing.  Both from
// bit_w4a4_quantized_amd/csrc/slots.h, without a GPU.
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <limits>

#include "../bit_w4a4_quantized_amd/csrc/slots.h"

using namespace svdq;

int main() {
  const int HUGE32 = std::numeric_limits<int>::max(), LOW32 = std::numeric_limits<int>::min();
  const int values[] = {LOW32, -1, 0, 7, 20, 40, 45, 46, HUGE32};
  int failures = 0, tiles = 0, owned = 0;
  for (const int a : values)
    for (const int b : values)
      for (const int c : values)
        for (const int d : values)
          for (const int group : {1, 2, 3, 8})
            for (const int R : {16, 32, 128}) {
              const int starts[] = {a, b, c, d}, tokens = 45, n = 3;
              const PagedBatch batch{nullptr, 0, 0, starts, nullptr, n};
              const int slots = tokens * group / R + n;
              for (int slot = 0; slot < slots; slot++)
                for (int i = 0; i < n; i++) {
                  const int s0 = start_of(batch, i, tokens), s1 = start_of(batch, i + 1, tokens);
                  const int rows = s1 > s0 ? (s1 - s0) * group : 0;
                  const int64_t first = first_slot(s0, group, R, i);
                  const int row0 = first_row_of(first, slot, R, rows);
                  tiles++;
                  if (row0 < 0) continue;
                  owned++;
                  for (int r = row0; r < row0 + R && r < rows; r++) {
                    const int token = s0 + r / group, head = r - r / group * group;
                    if (token < s0 || token >= s1 || head < 0 || head >= group) failures++;
                  }
                  if (row0 >= rows || slot < first) failures++;
                }
              // starts in order: every row of every sequence has a slot
              if (a <= b && b <= c && c <= d)
                for (int i = 0; i < n; i++) {
                  const int s0 = start_of(batch, i, tokens), s1 = start_of(batch, i + 1, tokens), rows = (s1 - s0) * group;
                  const int64_t first = first_slot(s0, group, R, i);
                  for (int r = 0; r < rows; r += R) {
                    const int64_t slot = first + r / R;
                    if (slot >= slots || first_row_of(first, (int)slot, R, rows) != r) failures++;
                    if (i + 1 < n && slot >= first_slot(s1, group, R, i + 1)) failures++;
                  }
                }
            }
  // quotients by numbers from the host
  uint32_t x = 1;
  auto any = [&](uint32_t below) { return (x = x * 1664525u + 1013904223u) % below; };
  for (int i = 0; i < 40000; i++) {
    const uint32_t d = i < 300 ? i + 1 : i < 400 ? 65536 - (i - 300) : 1 + any(65536), most = (1u << 31) + 255;
    const uint32_t q = any(most / d + 1) * d;
    for (const uint32_t n : {0u, d - 1, d, q, q - (q > 0), q + d - 1 < most ? q + d - 1 : q, most, any(most)})
      if (group_quotient(n, d, group_inverse((int)d)) != n / d) failures++;
  }
  for (uint32_t d = 2; d <= 128; d++)
    for (int i = 0; i < 2000; i++) {
      const uint32_t most = (1u << 25) + 127, q = any(most / d) * d;
      for (const uint32_t n : {0u, d - 1, d, q, q + d - 1, q - (q > 0), most, most - 127, any(most)})
        if (high_product(n, parts_inverse((int)d)) != n / d) failures++;
    }
  std::printf("%s: %d failure(s), %d of %d tiles with rows\n", failures ? "FAILED" : "OK", failures, owned, tiles);
  return failures ? 1 : 0;
}
