// C-ABI layer of the operators around a paged cache (include/svdq.h): host-side argument validation and
// kernel launches.  Every check happens before any HIP call; no exception leaves this file.
#include <math.h>

#include "../../include/svdq.h"
#include "paged.h"

using namespace svdq;

namespace {

constexpr int kMaxDim = 1 << 24;
constexpr int64_t kMaxStride = (int64_t)1 << 40;     // elements: keeps every index product below 2^63
constexpr int kMaxHeads = 1 << 16;
constexpr int kMaxHeadDim = 256;

inline bool is16(int t) { return t == SVDQ_TYPE_F16 || t == SVDQ_TYPE_BF16; }
inline bool is8(int t) { return t == SVDQ_TYPE_INT8 || t == SVDQ_TYPE_E4M3; }
inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }
inline bool eps_ok(float e) { return isfinite(e) && e > 0.f; }
inline bool scale_ok(float s) { return s >= 0x1p-126f && s <= 0x1p126f; }     // its product with log2(e) is a normal number
inline bool power_of_two(int n) { return n > 0 && (n & (n - 1)) == 0; }

// Tiles of at least 16 rows: what 32-bit numbers of tiles and of their parts hold.
inline bool tiles_ok(int tokens, int heads, int kv_heads, int sequences) {
  return ((int64_t)tokens * (heads / kv_heads) / 16 + sequences) * kv_heads <= 1 << 24;
}

svdq_status map_launch(hipError_t e) {
  if (e == hipSuccess) return SVDQ_OK;
  if (e == hipErrorInvalidConfiguration) return SVDQ_ERR_SHAPE;   // !launchable
  if (e == hipErrorNoBinaryForGpu || e == hipErrorInvalidDeviceFunction) return SVDQ_ERR_DEVICE;
  return SVDQ_ERR_LAUNCH;
}

// Sizes, types and strides; `type`: of the step's tokens, which a 16-bit cache must have, or -1.
svdq_status check_sizes(const svdq_paged_cache* c, const svdq_paged_batch* b, int type) {
  if (!c || !b) return SVDQ_ERR_NULL;
  if ((!is16(c->type) && !is8(c->type)) || (type >= 0 && is16(c->type) && (int)c->type != type)) return SVDQ_ERR_FORMAT;
  if (c->pages < 0 || c->pages > 0x7FFFFFFF || !power_of_two(c->page_size) || c->page_size > 1 << 16) return SVDQ_ERR_SHAPE;
  if (c->heads < 1 || c->heads > kMaxHeads || c->dim < 8 || c->dim > kMaxHeadDim) return SVDQ_ERR_SHAPE;
  const int each = is16(c->type) ? 8 : 16;           // elements of 16 bytes
  if (c->dim % each) return SVDQ_ERR_SHAPE;
  for (const int64_t s : {c->page_stride, c->token_stride, c->head_stride})
    if (!stride_ok(s) || s % each) return SVDQ_ERR_SHAPE;
  if (is8(c->type))
    for (const int64_t s : {c->scale_page_stride, c->scale_token_stride, c->scale_head_stride})
      if (!stride_ok(s)) return SVDQ_ERR_SHAPE;
  if (b->sequences < 0 || b->sequences > kMaxDim || b->table_width < 0 || !stride_ok(b->table_stride)) return SVDQ_ERR_SHAPE;
  if ((int64_t)b->table_width * c->page_size > (int64_t)1 << 30) return SVDQ_ERR_SHAPE;
  return SVDQ_OK;
}

svdq_status check_pointers(const svdq_paged_cache& c, const svdq_paged_batch& b) {
  if (b.sequences > 0 && (!b.starts || !b.context || (b.table_width > 0 && !b.page_table))) return SVDQ_ERR_NULL;
  if (!aligned(b.starts, 4) || !aligned(b.context, 4) || !aligned(b.page_table, 4)) return SVDQ_ERR_ALIGN;
  if (c.pages > 0 && (!c.k || !c.v || (is8(c.type) && (!c.k_scales || !c.v_scales)))) return SVDQ_ERR_NULL;
  if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.k_scales, 4) || !aligned(c.v_scales, 4)) return SVDQ_ERR_ALIGN;
  return SVDQ_OK;
}

PagedCache cache_of(const svdq_paged_cache& c) {
  int shift = 0;
  while (1 << shift < c.page_size) shift++;
  return PagedCache{c.k, c.v, c.k_scales, c.v_scales, c.type, (int)c.pages, shift, c.heads, c.dim,
                    c.page_stride, c.token_stride, c.head_stride,
                    c.scale_page_stride, c.scale_token_stride, c.scale_head_stride};
}

PagedBatch batch_of(const svdq_paged_batch& b) {
  return PagedBatch{b.page_table, b.table_stride, b.table_width, b.starts, b.context, b.sequences};
}

}  // namespace

extern "C" {

svdq_status svdq_rope_append(const svdq_paged_cache* cache, const svdq_paged_batch* batch, const svdq_rope_operand* q,
                             const svdq_rope_operand* k, const void* v, int64_t v_token, int64_t v_head, int tokens,
                             svdq_type type, const void* positions, int positions_fp32, const float* inv_freq, int axes,
                             const int* axis_pairs, int halves, float eps, void* stream) {
  if (!is16(type)) return SVDQ_ERR_FORMAT;
  svdq_status st = check_sizes(cache, batch, type);
  if (st != SVDQ_OK) return st;
  if (!k || !axis_pairs) return SVDQ_ERR_NULL;
  if (tokens < 0 || tokens > kMaxDim || axes < 1 || axes > kMaxRopeAxes) return SVDQ_ERR_SHAPE;
  if (k->heads != cache->heads || !stride_ok(v_token) || !stride_ok(v_head)) return SVDQ_ERR_SHAPE;
  AppendArgs a{};
  RopeArgs& r = a.r;
  for (int i = 0; i < axes; i++) {
    if (axis_pairs[i] < 0 || axis_pairs[i] > cache->dim) return SVDQ_ERR_SHAPE;
    r.pairs += axis_pairs[i];
    r.end[i] = r.pairs;
  }
  for (int i = axes; i < kMaxRopeAxes; i++) r.end[i] = r.pairs;
  if (r.pairs < 1 || 2 * r.pairs > cache->dim) return SVDQ_ERR_SHAPE;
  int64_t heads = (int64_t)2 * cache->heads;
  for (const svdq_rope_operand* o : {q, k}) {
    if (!o) continue;
    if (o->heads < 1 || o->heads > kMaxHeads) return SVDQ_ERR_SHAPE;
    for (const int64_t s : {o->in_token, o->in_head})
      if (!stride_ok(s)) return SVDQ_ERR_SHAPE;
    if (o == q && (!stride_ok(o->out_token) || !stride_ok(o->out_head))) return SVDQ_ERR_SHAPE;
    if (o->weight && !eps_ok(eps)) return SVDQ_ERR_SHAPE;
    if (o == q) heads += o->heads;
  }
  if (tokens * heads >= (int64_t)1 << 31) return SVDQ_ERR_SHAPE;
  if (tokens == 0) return SVDQ_OK;
  if (!positions || !inv_freq || !k->in || !v || (q && (!q->in || !q->out))) return SVDQ_ERR_NULL;
  st = check_pointers(*cache, *batch);
  if (st != SVDQ_OK) return st;
  if (!aligned(positions, 4) || !aligned(inv_freq, 4) || !aligned(k->in, 2) || !aligned(v, 2) || !aligned(k->weight, 4))
    return SVDQ_ERR_ALIGN;
  if (q && (!aligned(q->in, 2) || !aligned(q->out, 2) || !aligned(q->weight, 4))) return SVDQ_ERR_ALIGN;
  if (q) r.op[0] = RopeOperand{q->in, q->out, q->weight, q->heads, 0, q->in_token, q->in_head, 0, q->out_token, q->out_head};
  r.op[1] = RopeOperand{k->in, nullptr, k->weight, k->heads, 0, k->in_token, k->in_head, 0, 0, 0};
  r.nops = 2;
  r.batch = 1;
  r.tokens = tokens;
  r.dim = cache->dim;
  r.type = type;
  r.positions = positions;
  r.pos_token = axes;
  r.pos_float = positions_fp32 != 0;
  r.inv_freq = inv_freq;
  r.axes = axes;
  r.halves = halves != 0;
  r.eps = eps;
  a.v = v;
  a.v_token = v_token;
  a.v_head = v_head;
  a.c = cache_of(*cache);
  a.b = batch_of(*batch);
  return map_launch(launch_append(a, static_cast<hipStream_t>(stream)));
}

svdq_status svdq_tree_attention(const svdq_paged_cache* cache, const svdq_paged_batch* batch, const void* q,
                                int64_t q_token, int64_t q_head, int heads, int tokens, svdq_type type, float scale,
                                const void* tree, int64_t tree_stride, int tree_width, void* out, int64_t out_token,
                                int64_t out_head, void* workspace, size_t workspace_bytes, void* stream) {
  if (!is16(type)) return SVDQ_ERR_FORMAT;
  svdq_status st = check_sizes(cache, batch, type);
  if (st != SVDQ_OK) return st;
  if (tokens < 0 || tokens > kMaxDim || heads < 1 || heads > kMaxHeads || heads % cache->heads) return SVDQ_ERR_SHAPE;
  if ((int64_t)tokens * heads >= (int64_t)1 << 31 || !scale_ok(scale)) return SVDQ_ERR_SHAPE;
  if (!tiles_ok(tokens, heads, cache->heads, batch->sequences)) return SVDQ_ERR_SHAPE;
  for (const int64_t s : {q_token, q_head, out_token, out_head})
    if (!stride_ok(s)) return SVDQ_ERR_SHAPE;
  if (tree && (!stride_ok(tree_stride) || tree_width < 0)) return SVDQ_ERR_SHAPE;
  if (tokens == 0 || batch->sequences == 0) return SVDQ_OK;
  if (!q || !out) return SVDQ_ERR_NULL;
  st = check_pointers(*cache, *batch);
  if (st != SVDQ_OK) return st;
  if (!aligned(q, 2) || !aligned(out, 2) || !aligned(workspace, 16)) return SVDQ_ERR_ALIGN;
  AttnArgs a{};
  a.c = cache_of(*cache);
  a.b = batch_of(*batch);
  a.q = q;
  a.q_token = q_token;
  a.q_head = q_head;
  a.o = out;
  a.o_token = out_token;
  a.o_head = out_head;
  a.tokens = tokens;
  a.heads = heads;
  a.group = heads / cache->heads;
  a.qbf = type == SVDQ_TYPE_BF16;
  a.scale = scale * 1.4426950408889634f;
  a.tree = static_cast<const uint8_t*>(tree);
  a.tree_stride = tree_stride;
  a.tree_width = tree_width;
  const AttnPlan p = attn_plan(batch->sequences, tokens, heads, cache->heads, cache->dim,
                               (int64_t)batch->table_width * cache->page_size, workspace ? workspace_bytes : 0);
  a.rows = p.rows;
  a.slots = p.slots;
  a.unit = p.unit;
  a.ids = p.ids;
  a.whole = p.whole;
  a.parts = p.parts;
  a.group_inverse = group_inverse(a.group);
  a.parts_inverse = p.parts > 1 ? parts_inverse(p.parts) : 0;
  a.part = static_cast<float*>(workspace);
  return map_launch(launch_attn(a, static_cast<hipStream_t>(stream)));
}

size_t svdq_tree_attention_workspace_bytes(int sequences, int tokens, int heads, int kv_heads, int dim, int table_width,
                                           int page_size) {
  if (sequences < 1 || tokens < 1 || kv_heads < 1 || heads < kv_heads || heads % kv_heads || heads > kMaxHeads ||
      tokens > kMaxDim || sequences > kMaxDim || dim < 8 || dim > kMaxHeadDim || table_width < 0 || page_size < 1 ||
      (int64_t)tokens * heads >= (int64_t)1 << 31 || (int64_t)table_width * page_size > (int64_t)1 << 30 ||
      !tiles_ok(tokens, heads, kv_heads, sequences))
    return 0;
  return attn_plan(sequences, tokens, heads, kv_heads, dim, (int64_t)table_width * page_size, ~(size_t)0).bytes;
}

svdq_status svdq_cache_keep(const svdq_paged_cache* cache, const svdq_paged_batch* batch, const int* path,
                            int64_t path_stride, int path_width, void* stream) {
  const svdq_status st = check_sizes(cache, batch, -1);
  if (st != SVDQ_OK) return st;
  if (path_width < 0 || path_width > 1 << 16 || !stride_ok(path_stride)) return SVDQ_ERR_SHAPE;
  if (path_width == 0 || batch->sequences == 0) return SVDQ_OK;
  if (!path) return SVDQ_ERR_NULL;
  if (!aligned(path, 4)) return SVDQ_ERR_ALIGN;
  const svdq_status pt = check_pointers(*cache, *batch);
  if (pt != SVDQ_OK) return pt;
  const KeepArgs a{cache_of(*cache), batch_of(*batch), path, path_stride, path_width};
  return map_launch(launch_keep(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
