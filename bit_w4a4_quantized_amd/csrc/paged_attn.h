// Shared by the attention kernels over a paged cache (k_attn_few.hip, k_attn_many.hip, k_attn_join.hip).
#pragma once
#include "paged.h"
#include "rope.h"

namespace svdq {
namespace attn {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// What the cache holds: the queries' own 16-bit type, or codes, which become fp16 (exactly: 8 bits and E4M3's
// range fit it), and so do the queries then.
enum Kind { C16, CI8, CE4 };

// A row's powers p_j are taken relative to 2^m, its products with V's scales (8-bit caches) relative to 2^(m + r), each
// for the row alone and from the keys that it sees.  A reference moves when a logit (for m + r: a product's logarithm)
// passes it by kSlack, and then only that row's: most tiles need no exchange between lanes and no rescaling, and what
// other rows see changes no bit of this one.  Logits are only ever subtracted from one another: a sum with a small number
// could lose it (logits have steps of 16 from 2^27 on).
//
// What becomes an fp16 operand lies high in its range: a reference is moved to kLand below the largest, which then is at
// 2^7 and stays below 2^15.  Operands 2^-21 of it keep all bits, smaller ones are off by 2^-32 of it (of 131071 keys 18
// nats below one other, whose value is 0, nothing was left with the largest at 1).
constexpr float kSlack = 8.f, kLand = 7.f;

// The row's largest logit of a tile against its reference; the factor of its sums.
template <bool LAND>
__device__ __forceinline__ float move_powers(float top, float& m) {
  constexpr float land = LAND ? kLand : 0.f;
  const float old = m;
  if (top - old > land + kSlack) m = top - land;       // the first tile: from minus infinity
  return m == old ? 1.f : __builtin_amdgcn_exp2f(old - m);
}
// The same for the products, after a move of m by `by`; vtop: the largest product's logarithm, less m.  r stays where
// 2^r and 2^-r are normal numbers: products so much smaller or larger than the powers are below or past the output's range.
__device__ __forceinline__ float move_products(float vtop, float by, float& r) {
  const float kept = r - by;
  r = fmaxf(kept, -120.f);
  if (vtop - r > kLand + kSlack) r = fminf(vtop - kLand, 126.f);
  return r == kept ? 1.f : __builtin_amdgcn_exp2f(kept - r);
}

// The largest of a wave's values, in every lane.
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp<0xB1>(v));
  v = fmaxf(v, dpp<0x4E>(v));
  v = fmaxf(v, dpp<0x141>(v));
  v = fmaxf(v, dpp<0x140>(v));
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}

template <bool BF>
__device__ __forceinline__ v4f mfma16(const v4u& x, const v4u& y, const v4f& z) {
  if (BF) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x), __builtin_bit_cast(v8bf, y), z, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, x), __builtin_bit_cast(v8h, y), z, 0, 0, 0);
}

// Eight codes of a piece of sixteen (its first half or second) as fp16.
template <int CK>
__device__ __forceinline__ v4u widen(const v4u& u, int second) {
  const uint32_t w[2] = {second ? u[2] : u[0], second ? u[3] : u[1]};
  v4u r;
#pragma unroll
  for (int i = 0; i < 2; i++) {
    if (CK == CE4) {
      r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[i], 1.0f, false));
      r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[i], 1.0f, true));
    } else {
      // code + 128 as the low byte of a half in [1024, 2048), whose steps are ones; 1152 off it is exact
      const uint32_t b = w[i] ^ 0x80808080u;
      const f16x2 off = {(_Float16)1152.f, (_Float16)1152.f};
      const f16x2 lo = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u)) - off;
      const f16x2 hi = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u)) - off;
      r[2 * i] = __builtin_bit_cast(uint32_t, lo);
      r[2 * i + 1] = __builtin_bit_cast(uint32_t, hi);
    }
  }
  return r;
}

// A piece of V (16-bit values) without its infinities and NaN, which 0 * infinity would bring to rows that do not
// see them; whether there were any.
template <bool BF>
__device__ __forceinline__ bool make_finite(v4u& u) {
  constexpr uint32_t e = BF ? 0x7F80u : 0x7C00u;
  bool r = false;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const bool lo = (u[i] & e) == e, hi = (u[i] >> 16 & e) == e;
    u[i] &= (lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u);
    r = r || lo || hi;
  }
  return r;
}

// A value of a row of the cache, without its scale.
template <bool BF, int CK>
__device__ __forceinline__ float one_value(const uint8_t* row, int at) {
  if (CK == CI8) return (float)reinterpret_cast<const int8_t*>(row)[at];
  if (CK == CE4) return __builtin_amdgcn_cvt_f32_fp8((int)row[at], 0);
  const uint32_t b = reinterpret_cast<const uint16_t*>(row)[at];
  return BF ? bf16_f32(b) : f16_f32(b);
}

// What a logit's sum of products is multiplied by is a.scale, apart in 8-bit caches: K's scales in LDS take a factor in
// [1, 2), the sums a power of two, whose products are not rounded.
__device__ __forceinline__ int scale_power(const AttnArgs& a) { return __builtin_amdgcn_frexp_expf(a.scale) - 1; }
__device__ __forceinline__ float scale_factor(const AttnArgs& a) { return __builtin_ldexpf(a.scale, -scale_power(a)); }
__device__ __forceinline__ float power_of_two(int e) { return __builtin_ldexpf(1.f, min(max(e, -126), 126)); }

// A row of bf16 queries (its pieces lie in every NEAR-th lane: 16 or 32) as fp16, divided by
// a power of two that brings its largest into [2^14, 2^15): exact for values down to 2^-28 of the largest and
// within 2^-39 of it below.  Returns the power.
template <int N, int NEAR>
__device__ __forceinline__ int queries_to_f16(v4u* q) {
  float top = 0.f;
#pragma unroll
  for (int s = 0; s < N; s++)
#pragma unroll
    for (int i = 0; i < 4; i++)
      top = fmaxf(top, fmaxf(__builtin_fabsf(bf16_f32(q[s][i] & 0xFFFFu)), __builtin_fabsf(bf16_f32(q[s][i] >> 16))));
  if (NEAR == 16) top = fmaxf(top, __shfl_xor(top, 16));
  top = fmaxf(top, __shfl_xor(top, 32));
  const int e = top > 0.f && top < INFINITY ? __builtin_amdgcn_frexp_expf(top) - 15 : 0;
#pragma unroll
  for (int s = 0; s < N; s++)
#pragma unroll
    for (int i = 0; i < 4; i++)
      q[s][i] = pack_f16(__builtin_ldexpf(bf16_f32(q[s][i] & 0xFFFFu), -e), __builtin_ldexpf(bf16_f32(q[s][i] >> 16), -e));
  return e;
}

// Four values of each of two blocks of a matrix in LDS, turned: among 16 lanes, lane 4 r + p points at values
// 4 p ... of row r and gets column lane % 16 of the four rows.
__device__ __forceinline__ v4u transposed(const uint16_t* x, const uint16_t* y) {
  typedef __attribute__((address_space(3))) s16x4 lds4;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)x), b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)y);
  const u32x2_t p = __builtin_bit_cast(u32x2_t, a), q = __builtin_bit_cast(u32x2_t, b);
  return v4u{p[0], p[1], q[0], q[1]};
}

constexpr int kManyRows = 128, kFewRows = 32;   // 16 or 32 where there are no more (32 of heads up to 128: registers)

// A launch has fewer than 2^32 threads along x: 2^24 tiles of few rows, the most there are, take two rows of the grid.
constexpr int kGridRow = 1 << 23;

__host__ __device__ inline int64_t blocks_of(const AttnArgs& a) {
  const int64_t tiles = (int64_t)a.slots * a.c.heads;
  return a.whole + (tiles - a.whole) * a.parts;
}

// A workgroup's share: rows row0 ... of a sequence (token * group + query head of the group), a cache head
// and keys begin ... end - 1.
struct Work {
  int seq, head;
  int s0, n, ctx, keys;                      // s0: first token; n: tokens; keys: context and tokens that have a slot
  int row0, rows, begin, end;
  int64_t id;                                // of its sums among all parts'; below 0: the tile has all its keys here

  // Whether token i of the sequence sees an existing key.
  __device__ __forceinline__ bool sees(const AttnArgs& a, int i, int key) const {
    const int j = key - ctx;
    if (j < 0) return true;
    if (!a.tree) return j <= i;
    return j < a.tree_width && a.tree[(int64_t)(s0 + i) * a.tree_stride + j];
  }
  // The same of keys key ... key + 3, a bit each.  Of a tree's row one load of four marks, moved to where it lies
  // within the row, and no branches: the loads of a lane's keys are in flight together.
  __device__ __forceinline__ uint32_t sees4(const AttnArgs& a, int i, int key) const {
    const int j = key - ctx;
    if (!a.tree) return (1u << min(max(i - j + 1, 0), 4)) - 1;
    uint32_t bits = 0;
    if (a.tree_width >= 4) {
      const int at = min(max(j, 0), a.tree_width - 4), by = 8 * min(max(j - at, -4), 4);
      uint32_t x;
      __builtin_memcpy(&x, a.tree + (int64_t)(s0 + i) * a.tree_stride + at, 4);
      x = (uint32_t)(by < 0 ? (uint64_t)x << -by : (uint64_t)x >> by);
      x |= x >> 4;                           // a mark is any value but 0
      x |= x >> 2;
      x |= x >> 1;
      x &= 0x01010101u;
      bits = (x | x >> 7 | x >> 14 | x >> 21) & 0xFu;
    } else {
      for (int e = 0; e < 4; e++)
        if (j + e >= 0 && j + e < a.tree_width && a.tree[(int64_t)(s0 + i) * a.tree_stride + j + e]) bits |= 1u << e;
    }
    return bits | ((1u << min(max(-j, 0), 4)) - 1);    // the context's
  }
};

__device__ __forceinline__ int keys_of(const AttnArgs& a, int ctx, int n) {
  return (int)min((int64_t)ctx + n, (int64_t)a.b.width << a.c.shift);
}

// The rows of a slot.  Sequence i has the slots from floor(starts[i] group / R) + i on: one more than it may need,
// found without a sum over the sequences.
template <int R>
__device__ __forceinline__ bool find_rows(const AttnArgs& a, int slot, Work& w) {
  int s1;
  if (a.b.n <= 64) {                         // one look, at all that is asked of the sequence
    const int i = min(__lane_id(), a.b.n - 1);
    const int from = start_of(a.b, i, a.tokens), to = start_of(a.b, i + 1, a.tokens), ctx = context_of(a.b, i);
    const int64_t first = first_slot(from, a.group, R, i);
    const int count = __popcll(__ballot((int)__lane_id() < a.b.n && first <= slot));
    if (count == 0) return false;
    w.seq = __builtin_amdgcn_readfirstlane(count - 1);
    w.s0 = __builtin_amdgcn_readlane(from, w.seq);
    s1 = __builtin_amdgcn_readlane(to, w.seq);
    w.ctx = __builtin_amdgcn_readlane(ctx, w.seq);
  } else {
    w.seq = __builtin_amdgcn_readfirstlane(
        last_below(a.b.n, slot, [&](int i) { return first_slot(start_of(a.b, i, a.tokens), a.group, R, i); }));
    if (w.seq < 0) return false;
    w.s0 = start_of(a.b, w.seq, a.tokens);
    s1 = start_of(a.b, w.seq + 1, a.tokens);
    w.ctx = context_of(a.b, w.seq);
  }
  w.n = max(0, s1 - w.s0);
  w.rows = w.n * a.group;
  w.row0 = first_row_of(first_slot(w.s0, a.group, R, w.seq), slot, R, w.rows);
  if (w.row0 < 0) return false;
  w.keys = keys_of(a, w.ctx, w.n);
  return true;
}
// Tiles are numbered heads first (those of a cache head on one XCD, which share rows of the cache where a
// sequence has several), then slots of rows, the last first: a chunk's last rows see the most keys.
template <int R>
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int tile, Work& w) {
  w.head = tile % a.c.heads;
  return find_rows<R>(a, a.slots - 1 - tile / a.c.heads, w);
}

// How a tile's keys are shared among its parts: keys up to `last`, `units` of a.unit, `each` of them a part (a table
// wider than the contexts leaves the last parts without any).  The quotients by numbers from the host: k_attn_join waits for
// them (by division 0.4 to 2 us a call).
struct Shares {
  int last, units, each;
};
template <int R>
__device__ __forceinline__ Shares share_keys(const AttnArgs& a, const Work& w, int parts) {
  Shares s;
  s.last = w.keys;
  if (!a.tree) {
    const int token = (int)group_quotient(w.row0 + R - 1, a.group, a.group_inverse);
    s.last = min(w.keys, w.ctx + min(token, w.n - 1) + 1);
  }
  s.units = a.unit == 32 ? (s.last + 31) >> 5 : (s.last + 63) >> 6;
  s.each = parts == 1 ? s.units : (int)high_product(s.units + parts - 1, a.parts_inverse);
  return s;
}

// The workgroup's tile, or part of one that has keys.
template <int R>
__device__ __forceinline__ bool cut_work(const AttnArgs& a, Work& w) {
  int id = blockIdx.x;
  if (R <= kFewRows) {
    id += blockIdx.y * kGridRow;
    // Eight slots' parts at a time, a head after the other: workgroups go round the eight XCDs, so that the heads of a
    // part meet on one of them.  They share the cache lines of scales (and of short rows).
    const int all = (int)blocks_of(a) / a.c.heads, g = id / (8 * a.c.heads), in = id - g * 8 * a.c.heads, m = min(8, all - 8 * g);
    const int head = in / m;
    id = (8 * g + in - head * m) * a.c.heads + head;
  }
  int tile = id, split = 0, parts = 1;
  w.id = -1;
  if (id >= a.whole) {
    const int cut = a.slots * a.c.heads - a.whole, u = id - a.whole;
    split = u / cut;
    parts = a.parts;
    tile = a.whole + u - split * cut;
    if (parts > 1) w.id = (int64_t)(tile - a.whole) * parts + split;
  }
  if (!find_tile<R>(a, tile, w)) return false;
  const Shares s = share_keys<R>(a, w, parts);
  w.begin = min(s.last, split * s.each * a.unit);
  w.end = min(s.last, w.begin + s.each * a.unit);
  return w.id < 0 || w.begin < w.end;
}

// A value of V of an existing slot, where it is an infinity or NaN (with its scale), else 0: what make_finite took
// from the rows that do see it.
template <bool BF, int CK>
__device__ __forceinline__ float infinite_value(const AttnArgs& a, const Work& w, int page, int slot, int d) {
  const int64_t in_page = slot & ((1 << a.c.shift) - 1);
  const int64_t at = page * a.c.page + in_page * a.c.token + w.head * a.c.head;
  float x = one_value<BF, CK>(static_cast<const uint8_t*>(a.c.v) + at * (CK == C16 ? 2 : 1), d);
  if (CK != C16) x *= a.c.vs[page * a.c.spage + in_page * a.c.stoken + w.head * a.c.shead];
  return __builtin_fabsf(x) < INFINITY ? 0.f : x;
}

// Where a row's result goes: the output where the tile has all its keys, else this part's sums.
struct Dest {
  uint16_t* out;
  float* sums;
  float* ml;
};
template <int R>
__device__ __forceinline__ Dest dest_of(const AttnArgs& a, const Work& w, int row) {
  if (w.id < 0) {
    const int r = w.row0 + row, i = r / a.group, t = w.s0 + i, h = w.head * a.group + r - i * a.group;
    return {static_cast<uint16_t*>(a.o) + (int64_t)t * a.o_token + (int64_t)h * a.o_head, nullptr, nullptr};
  }
  return {nullptr, a.part + (w.id * R + row) * a.c.dim, a.part + a.ids * R * a.c.dim + (w.id * R + row) * 2};
}
// Four of its values, from d on, with the row's maximum and sum.
__device__ __forceinline__ void put(const Dest& to, bool bf, int d, const v4f& o, float m, float sum) {
  if (to.out) {
    const float f = sum == 0.f ? 0.f : 1.f / sum;      // a row that sees nothing is zeros
    const uint32_t x[2] = {pack16(o[0] * f, o[1] * f, bf), pack16(o[2] * f, o[3] * f, bf)};
    __builtin_memcpy(to.out + d, x, 8);
    return;
  }
  *reinterpret_cast<v4f*>(to.sums + d) = o;
  if (d == 0) {
    to.ml[0] = m;
    to.ml[1] = sum;
  }
}

hipError_t launch_few(const AttnArgs& a, hipStream_t s);
hipError_t launch_many(const AttnArgs& a, hipStream_t s);

}  // namespace attn
}  // namespace svdq
