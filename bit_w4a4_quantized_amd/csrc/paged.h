// Shared by the operators around a paged cache of keys and values (cache_api.hip, k_append.hip, paged_attn.h):
// the argument structs cache_api.hip fills, and how a kernel finds a token's sequence.
#pragma once
#include "block_ops.h"
#include "slots.h"

namespace svdq {

constexpr float kTiny = 0x1p-100f;           // floor of a head's absolute maximum: zeros get codes 0 and a finite scale

struct AppendArgs {
  RopeArgs r;                                // op[0] queries (heads 0: none), op[1] keys (out unused)
  const void* v; int64_t v_token, v_head;
  PagedCache c; PagedBatch b;
};
hipError_t launch_append(const AppendArgs& a, hipStream_t s);

struct KeepArgs {
  PagedCache c; PagedBatch b;
  const int* path; int64_t path_stride; int path_width;
};
hipError_t launch_keep(const KeepArgs& a, hipStream_t s);

struct AttnArgs {
  PagedCache c; PagedBatch b;
  const void* q; int64_t q_token, q_head;
  void* o; int64_t o_token, o_head;
  int tokens, heads, group, qbf;             // group: query heads a cache head; qbf: q and o are bf16
  float scale;                               // times log2(e)
  const uint8_t* tree; int64_t tree_stride; int tree_width;
  // A tile is `rows` rows of a sequence and cache head; its number is slot * cache heads + head.  The first
  // `whole` tiles take all their keys at once, the others are cut into `parts` each, of whole units of `unit` keys, and
  // joined afterwards.
  int rows, slots, unit, whole, parts;
  uint32_t group_inverse, parts_inverse;     // of group, and of parts past 1 (slots.h)
  int64_t ids;                               // of parts
  float* part;                               // fp32 [ids][rows][dim] sums, then [ids][rows][2]
};
// How a step's tiles are cut, for workspaces of at most `room` bytes.  reach: keys that the table can hold.
struct AttnPlan {
  int rows, slots, unit, whole, parts;
  int64_t ids;
  size_t bytes;
};
AttnPlan attn_plan(int sequences, int tokens, int heads, int kv_heads, int dim, int64_t reach, size_t room);
hipError_t launch_attn(const AttnArgs& a, hipStream_t s);

// The last i in [0, n) with f(i) <= target, for f that never falls; -1 if there is none.  The wave looks
// at 64 places at once, so that 4096 sequences take two loads' time.
template <typename F>
__device__ __forceinline__ int last_below(int n, int64_t target, F f) {
  const int lane = __lane_id();
  int lo = 0, len = n;
  for (;;) {
    const int step = (len + 63) / 64;
    const int i = lo + lane * step;
    const bool in = lane * step < len && f(min(i, n - 1)) <= target;
    const int count = __popcll(__ballot(in));
    if (count == 0) return lo - 1;           // only in the first turn: later ones begin at a place that holds
    lo += (count - 1) * step;
    if (step == 1) return lo;
    len = min(step, n - lo);
  }
}

}  // namespace svdq
