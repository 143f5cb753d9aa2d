// Which rows of attention a slot takes (bit_w4a4_quantized_amd/csrc/slots.h), for starts that hold anything: whatever
// sequence is found for a slot, its rows are tokens and heads that there are.  Without a GPU.
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
  std::printf("%s: %d failure(s), %d of %d tiles with rows\n", failures ? "FAILED" : "OK", failures, owned, tiles);
  return failures ? 1 : 0;
}
