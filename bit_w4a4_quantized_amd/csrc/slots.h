// Where a sequence's tokens lie in a paged cache.  Everything here that the host cannot see (a batch's starts,
// contexts and page table) may hold anything: starts are taken within the tokens there are, contexts within 0
// and 2^30, and a slot whose column or page does not exist is absent (never written, hidden from attention).
// Plain C++, for kernels and for tests without a GPU.
#pragma once
#include <stdint.h>

#ifdef __HIP__
#define SVDQ_BOTH __host__ __device__
#else
#define SVDQ_BOTH
#endif

namespace svdq {

constexpr int kMaxContext = 1 << 30;

struct PagedCache {
  void* k; void* v; float* ks; float* vs; int type;
  int pages, shift, heads, dim;              // 2^shift tokens a page
  int64_t page, token, head;                 // strides in elements, of k and v
  int64_t spage, stoken, shead;              // of ks and vs
};

struct PagedBatch {
  const int* table; int64_t stride; int width;
  const int* starts; const int* context; int n;
};

SVDQ_BOTH inline int within(int v, int most) { return v < 0 ? 0 : v > most ? most : v; }
SVDQ_BOTH inline int start_of(const PagedBatch& b, int i, int tokens) { return within(b.starts[i], tokens); }
SVDQ_BOTH inline int context_of(const PagedBatch& b, int i) { return within(b.context[i], kMaxContext); }

// What the table says of a sequence's slot, -1 past its width; and that as a page, -1 where it is none.  Apart, so
// that a kernel can look a tile ahead without waiting for the answer.
SVDQ_BOTH inline int entry_of(const PagedBatch& b, const PagedCache& c, int seq, int slot) {
  const int col = slot >> c.shift;
  return col < b.width ? b.table[seq * b.stride + col] : -1;
}
SVDQ_BOTH inline int as_page(const PagedCache& c, int entry) { return (unsigned)entry < (unsigned)c.pages ? entry : -1; }
SVDQ_BOTH inline int page_of(const PagedBatch& b, const PagedCache& c, int seq, int slot) {
  return as_page(c, entry_of(b, c, seq, slot));
}

// Attention's rows (a token times `group` query heads) in slots of R.  Sequence i has the slots from first_slot on, one
// more than it may need.  The row that a slot begins with, of a sequence of `rows` that was found for it: -1 where it has
// none.  Starts that fall can find a sequence whose first slot lies behind this one.
SVDQ_BOTH inline int64_t first_slot(int start, int group, int R, int i) { return (int64_t)start * group / R + i; }
SVDQ_BOTH inline int first_row_of(int64_t first, int slot, int R, int rows) {
  const int64_t row = (slot - first) * R;
  return row < 0 || row >= rows ? -1 : (int)row;
}

// Quotients by a number d that the host knows, without a division.  group_inverse: of any x below 2^31 + 2^8 by d up to
// 2^16; the product is the quotient or one less.  parts_inverse: of x up to 2^25 + 127 by d in 2 ... 128; the excess
// of the inverse, below d, adds less than one d-th.
SVDQ_BOTH inline uint32_t high_product(uint32_t x, uint32_t y) { return (uint32_t)((uint64_t)x * y >> 32); }
inline uint32_t group_inverse(int d) { return d == 1 ? 0xFFFFFFFFu : (uint32_t)(((uint64_t)1 << 32) / d); }
inline uint32_t parts_inverse(int d) { return (uint32_t)((((uint64_t)1 << 32) + d - 1) / d); }
SVDQ_BOTH inline uint32_t group_quotient(uint32_t x, uint32_t d, uint32_t inverse) {
  const uint32_t q = high_product(x, inverse);
  return x - q * d >= d ? q + 1 : q;
}

}  // namespace svdq
