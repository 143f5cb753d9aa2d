// A step's tokens into a paged cache, and the accepted ones of a draft moved together.
//
// svdq_rope_append, of each token's heads (see k_rope.hip for the turning):
//   queries  q' = rnd(turn(norm(q)));
//   keys     turn(norm(k)) to slot context[b] + i of the token's sequence b, rounded once: to the cache's
//            16-bit type, or to codes rnd(u * (qmax / a)) with the scale a / qmax, a = max(max|u|, 2^-100)
//            over the head (qmax 127 or 448);  values the same way, neither normed nor turned.
// Latency bounds few tokens: everything is one launch, and a wave loads its heads before it looks for their sequence
// and page (64 tokens of 32 + 16 heads of 128 5.7 us).  Many are bound by HBM and the vector unit together: 16384 tokens
// of 24 + 48 heads of 128 to E4M3 codes, 509 MB, take 130 us, 3.9 TB/s of the 4.9 that a large copy reaches, with the
// vector unit busy for three quarters of it (the norm, the angles, codes).  Three heads a lane group instead of two: an
// eighth fewer instructions, 135 us (four waves a SIMD for five).
#include "paged.h"
#include "rope.h"

namespace svdq {

namespace {

__device__ __forceinline__ float group_max(float v, int lanes) {
  if (lanes > 1) v = fmaxf(v, dpp<0xB1>(v));
  if (lanes > 2) v = fmaxf(v, dpp<0x4E>(v));
  if (lanes > 4) v = fmaxf(v, dpp<0x141>(v));
  if (lanes > 8) v = fmaxf(v, dpp<0x140>(v));
  for (int m = 16; m < lanes; m *= 2) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}

// Eight codes of values times mul.
__device__ __forceinline__ uint2 codes8(const float* y, float mul, int type) {
  uint32_t c[2];
  if (type == T_INT8) {
#pragma unroll
    for (int w = 0; w < 2; w++) {
      c[w] = 0;
#pragma unroll
      for (int e = 0; e < 4; e++) c[w] |= ((uint32_t)(int)__builtin_rintf(y[4 * w + e] * mul) & 0xFFu) << (8 * e);
    }
  } else {
#pragma unroll
    for (int w = 0; w < 2; w++) {
      const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * w] * mul, y[4 * w + 1] * mul, 0, false);
      c[w] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * w + 2] * mul, y[4 * w + 3] * mul, lo, true);
    }
  }
  return make_uint2(c[0], c[1]);
}

// Where a token's keys and values go: the element offset of head 0 of its slot, of the scales', or -1.
struct Place {
  int64_t at, sat;
};
__device__ __forceinline__ Place place_of(const AppendArgs& a, int seq, int slot) {
  const int id = page_of(a.b, a.c, seq, slot);
  if (id < 0) return {-1, -1};
  const int64_t off = slot & ((1 << a.c.shift) - 1);
  return {id * a.c.page + off * a.c.token, id * a.c.spage + off * a.c.stoken};
}
// The slot of token t, whose sequence is `seq` if that holds it; -1: the token belongs to none.
__device__ __forceinline__ int slot_of(const AppendArgs& a, int seq, int t) {
  if (seq < 0) return -1;
  const int s0 = start_of(a.b, seq, a.r.tokens), s1 = start_of(a.b, seq + 1, a.r.tokens);
  return t >= s0 && t < s1 ? context_of(a.b, seq) + (t - s0) : -1;
}

__device__ __forceinline__ float qmax(int type) { return type == T_INT8 ? 127.f : 448.f; }

enum Form { ADJACENT, PARTIAL, HALVES, HALVES_PARTIAL };     // as in k_rope.hip, and halves of a part of the head

struct Split {
  int tw, batches, waves, heads;             // tokens a wave; parts of a token's heads; waves; heads
};
struct Splits {
  Split of[2];                               // queries; keys and then values
};

// 16-byte pieces, a lane two pieces of a head, as k_rope has them; U heads a lane group.  Workgroups of
// keys and values come first: they have the longer chain of loads.
template <bool BF, Form FORM, int U>
__global__ void __launch_bounds__(256) k_append(AppendArgs a, int lanes, Splits sp) {
  __shared__ __attribute__((aligned(16))) float table[4][2][512];   // cosines and sines of each wave's tokens
  const RopeArgs& r = a.r;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int kv_blocks = (sp.of[1].waves + 3) / 4;
  const int which = (int)blockIdx.x < kv_blocks;
  const int id = __builtin_amdgcn_readfirstlane(((int)blockIdx.x - (which ? 0 : kv_blocks)) * 4 + wave);
  const Split& w_ = sp.of[which];
  if (id >= w_.waves) return;                // whole waves; no workgroup barrier below
  const RopeOperand& o = r.op[which];
  const int groups = 64 / lanes, j = lane % lanes, g = lane / lanes;
  const int nv = r.dim / 8, half = (nv + 1) / 2, pairs = r.dim / 2;
  // The lane's two pieces: half a head apart, of a part of the head that halves turn half of that apart, and behind it
  // half of what is left.
  int first_piece = j, second_piece = j + half;
  if (FORM == HALVES_PARTIAL) {
    const int apart = r.pairs / 8;
    if (j < apart) {
      second_piece = j + apart;
    } else {
      first_piece = j + apart;
      second_piece = first_piece + (nv - 2 * apart + 1) / 2;
    }
  }
  const bool in0 = j < half, in1 = j < half && second_piece < nv;
  const int part = id % w_.batches, t0 = id / w_.batches * w_.tw;
  const int nt = min(w_.tw, r.tokens - t0);
  const int first = part * U * groups, last = min(nt * w_.heads, first + U * groups);
  uint4 raw[U][2];
  int tl[U], hd[U];
  bool is_v[U];
#pragma unroll
  for (int i = 0; i < U; i++) {
    const int u = first + i * groups + g;
    raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
    tl[i] = w_.tw > 1 ? u / w_.heads : 0;
    hd[i] = u < last ? u - tl[i] * w_.heads : -1;
    if (hd[i] < 0) tl[i] = 0;
    is_v[i] = which && hd[i] >= a.c.heads;
    if (hd[i] >= 0) {
      const int64_t t = t0 + tl[i];
      if (is_v[i]) hd[i] -= a.c.heads;
      const uint16_t* p = is_v[i] ? static_cast<const uint16_t*>(a.v) + t * a.v_token + hd[i] * a.v_head
                                  : static_cast<const uint16_t*>(o.in) + t * o.in_token + hd[i] * o.in_head;
      if (in0) raw[i][0] = *reinterpret_cast<const uint4*>(p + first_piece * 8);
      if (in1) raw[i][1] = *reinterpret_cast<const uint4*>(p + second_piece * 8);
    }
  }
  int seq = 0;
  if (which) seq = last_below(a.b.n, t0, [&](int i) { return (int64_t)start_of(a.b, i, r.tokens); });
  // pairs past the turned ones get the identity (not used: below)
  for (int i = lane; i < nt * pairs; i += 64) {
    const int tl_ = w_.tw > 1 ? i / pairs : 0, p = i - tl_ * pairs;
    float c = 1.f, s = 0.f;
    if (p < r.pairs) pair_cos_sin(r, (int64_t)(t0 + tl_) * r.pos_token, p, &c, &s);
    table[wave][0][i] = c;
    table[wave][1][i] = s;
  }
  const bool norm = o.weight != nullptr;
  float w[2][8];
  if (norm) {
#pragma unroll
    for (int v = 0; v < 2; v++) __builtin_memcpy(w[v], o.weight + min((v ? second_piece : first_piece) * 8, r.dim - 8), 32);
  }
  Place place[U];
  if (which) {
#pragma unroll
    for (int i = 0; i < U; i++) {
      int at = seq;
      if (w_.tw > 1)
        while (at + 1 < a.b.n && start_of(a.b, at + 1, r.tokens) <= t0 + tl[i]) at++;
      const int slot = hd[i] < 0 ? -1 : slot_of(a, at, t0 + tl[i]);
      place[i] = slot < 0 ? Place{-1, -1} : place_of(a, at, slot);
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < U; i++) {
    float u[2][8], y[2][8];
    unpack8(raw[i][0], BF, u[0]);
    unpack8(raw[i][1], BF, u[1]);
    if (norm) {                              // values take part in the lanes' sums and keep their own
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; e++) ss += u[0][e] * u[0][e] + u[1][e] * u[1][e];
      ss = group_sum(ss, lanes);
      float rstd = root(r, ss);
      if (BF && __any(!(ss < INFINITY))) {
        float sd = 0.f;
#pragma unroll
        for (int e = 0; e < 8; e++) sd += small_square(u[0][e]) + small_square(u[1][e]);
        sd = group_sum(sd, lanes);
        if (!(ss < INFINITY)) rstd = root_down(r, sd);
      }
      if (!is_v[i]) {
#pragma unroll
        for (int v = 0; v < 2; v++)
#pragma unroll
          for (int e = 0; e < 8; e++) u[v][e] = u[v][e] * rstd * w[v][e];
      }
    }
    if (is_v[i]) {
#pragma unroll
      for (int v = 0; v < 2; v++)
#pragma unroll
        for (int e = 0; e < 8; e++) y[v][e] = u[v][e];
    } else {
      float c[8], s[8];
      // the lane's eight pairs: of its two pieces (adjacent), or between them (half apart)
#pragma unroll
      for (int v = 0; v < 2; v++) {
        const int p = tl[i] * pairs + min(FORM >= HALVES ? j * 8 + v * 4 : (j + v * half) * 4, pairs - 4);
        *reinterpret_cast<float4*>(c + 4 * v) = *reinterpret_cast<const float4*>(&table[wave][0][p]);
        *reinterpret_cast<float4*>(s + 4 * v) = *reinterpret_cast<const float4*>(&table[wave][1][p]);
      }
      if (FORM >= HALVES) {
#pragma unroll
        for (int e = 0; e < 8; e++) {
          y[0][e] = u[0][e] * c[e] - u[1][e] * s[e];
          y[1][e] = u[0][e] * s[e] + u[1][e] * c[e];
        }
      } else {
#pragma unroll
        for (int v = 0; v < 2; v++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const float cc = c[4 * v + e], sn = s[4 * v + e];
            y[v][2 * e] = u[v][2 * e] * cc - u[v][2 * e + 1] * sn;
            y[v][2 * e + 1] = u[v][2 * e] * sn + u[v][2 * e + 1] * cc;
          }
      }
      // values behind the pairs as they are: turned by the identity, an infinity or NaN would reach its neighbour
      if (FORM == PARTIAL) {
#pragma unroll
        for (int v = 0; v < 2; v++)
#pragma unroll
          for (int e = 0; e < 8; e++)
            if ((j + v * half) * 4 + e / 2 >= r.pairs) y[v][e] = u[v][e];
      }
      if (FORM == HALVES_PARTIAL) {
#pragma unroll
        for (int v = 0; v < 2; v++)
#pragma unroll
          for (int e = 0; e < 8; e++)
            if (j >= r.pairs / 8) y[v][e] = u[v][e];
      }
    }
    if (!which) {
      if (hd[i] < 0) continue;
      uint16_t* out = static_cast<uint16_t*>(o.out) + (int64_t)(t0 + tl[i]) * o.out_token + hd[i] * o.out_head;
      if (in0) stream16(out + first_piece * 8, pack8(y[0], BF));
      if (in1) stream16(out + second_piece * 8, pack8(y[1], BF));
    } else if (a.c.type == T_F16 || a.c.type == T_BF16) {
      if (place[i].at < 0) continue;
      uint16_t* out = static_cast<uint16_t*>(is_v[i] ? a.c.v : a.c.k) + place[i].at + hd[i] * a.c.head;
      // nontemporal as the queries' (k_rope.hip)
      if (in0) stream16(out + first_piece * 8, is_v[i] ? raw[i][0] : pack8(y[0], BF));
      if (in1) stream16(out + second_piece * 8, is_v[i] ? raw[i][1] : pack8(y[1], BF));
    } else {
      // lanes past a head's end hold zeros turned by the last pairs: zeros
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 8; e++) {
        if (in0) top = fmaxf(top, __builtin_fabsf(y[0][e]));
        if (in1) top = fmaxf(top, __builtin_fabsf(y[1][e]));
      }
      top = fmaxf(group_max(top, lanes), kTiny);
      if (place[i].at < 0) continue;
      const float mul = qmax(a.c.type) / top;
      uint8_t* out = static_cast<uint8_t*>(is_v[i] ? a.c.v : a.c.k) + place[i].at + hd[i] * a.c.head;
      if (in0) *reinterpret_cast<uint2*>(out + first_piece * 8) = codes8(y[0], mul, a.c.type);
      if (in1) *reinterpret_cast<uint2*>(out + second_piece * 8) = codes8(y[1], mul, a.c.type);
      if (j == 0) (is_v[i] ? a.c.vs : a.c.ks)[place[i].sat + hd[i] * a.c.shead] = top / qmax(a.c.type);
    }
  }
}

// Any pairing, stride and alignment of the step's tokens: one wave a head, its values in LDS.
template <bool BF>
__global__ void __launch_bounds__(256) k_append_any(AppendArgs a, int64_t units) {
  __shared__ __attribute__((aligned(16))) float head[4][256];
  const RopeArgs& r = a.r;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (unit >= units) return;                 // whole waves; no workgroup barrier below
  const int lane = threadIdx.x & 63;
  float* x = head[threadIdx.x >> 6];
  const int heads = r.op[0].heads + 2 * a.c.heads;
  const int t = (int)(unit / heads);
  int hd = (int)(unit - (int64_t)t * heads);
  const bool is_q = hd < r.op[0].heads;
  if (!is_q) hd -= r.op[0].heads;
  const bool is_v = !is_q && hd >= a.c.heads;
  if (is_v) hd -= a.c.heads;
  const RopeOperand& o = r.op[is_q ? 0 : 1];
  const uint16_t* in = is_v ? static_cast<const uint16_t*>(a.v) + t * a.v_token + hd * a.v_head
                            : static_cast<const uint16_t*>(o.in) + t * o.in_token + hd * o.in_head;
  float ss = 0.f, sd = 0.f;
  for (int d = lane; d < r.dim; d += 64) {
    const float v = load16(in, d, BF);
    x[d] = v;
    ss += v * v;
    sd += small_square(v);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (!is_v) {
    ss = group_sum(ss, 64);
    sd = group_sum(sd, 64);
    const float rstd = !o.weight ? 1.f : ss < INFINITY ? root(r, ss) : root_down(r, sd);
    auto val = [&](int d) { return o.weight ? x[d] * rstd * o.weight[d] : x[d]; };
    // a value belongs to one lane alone from here to the next barrier
    for (int p = lane; p < r.pairs; p += 64) {
      float c, s;
      pair_cos_sin(r, (int64_t)t * r.pos_token, p, &c, &s);
      const int i = r.halves ? p : 2 * p, k = r.halves ? p + r.pairs : 2 * p + 1;
      const float u = val(i), w = val(k);
      x[i] = u * c - w * s;
      x[k] = u * s + w * c;
    }
    for (int d = 2 * r.pairs + lane; d < r.dim; d += 64) x[d] = val(d);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  if (is_q) {
    uint16_t* out = static_cast<uint16_t*>(o.out) + t * o.out_token + hd * o.out_head;
    for (int d = lane; d < r.dim; d += 64) store16(out, d, x[d], BF);
    return;
  }
  const int seq = last_below(a.b.n, t, [&](int i) { return (int64_t)start_of(a.b, i, r.tokens); });
  const int slot = slot_of(a, seq, t);
  const Place pl = slot < 0 ? Place{-1, -1} : place_of(a, seq, slot);
  if (pl.at < 0) return;                     // the same in every lane
  float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, top = 0.f;
  const bool have = lane * 8 < r.dim;        // dim is a multiple of 8
  if (have) {
#pragma unroll
    for (int e = 0; e < 8; e++) {
      y[e] = x[lane * 8 + e];
      top = fmaxf(top, __builtin_fabsf(y[e]));
    }
  }
  const int64_t at = pl.at + hd * a.c.head + lane * 8;
  void* base = is_v ? a.c.v : a.c.k;
  if (a.c.type == T_F16 || a.c.type == T_BF16) {
    if (have) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = pack8(y, BF);
    return;
  }
  top = fmaxf(group_max(top, 64), kTiny);
  if (have) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + at) = codes8(y, qmax(a.c.type) / top, a.c.type);
  if (lane == 0) (is_v ? a.c.vs : a.c.ks)[pl.sat + hd * a.c.shead] = top / qmax(a.c.type);
}

bool wide(const AppendArgs& a) {
  const RopeArgs& r = a.r;
  if (r.halves && r.pairs % 8) return false;
  uintptr_t p = reinterpret_cast<uintptr_t>(r.op[1].in) | reinterpret_cast<uintptr_t>(a.v);
  int64_t st = r.op[1].in_token | r.op[1].in_head | a.v_token | a.v_head;
  if (r.op[0].heads) {
    p |= reinterpret_cast<uintptr_t>(r.op[0].in) | reinterpret_cast<uintptr_t>(r.op[0].out);
    st |= r.op[0].in_token | r.op[0].in_head | r.op[0].out_token | r.op[0].out_head;
  }
  return p % 16 == 0 && st % 8 == 0;
}

// Each kept token to its place: slot context + i takes slot context + path[i].  A thread has one piece of a
// head's keys or values (or a scale) over the whole path, in the path's order and kKeepAhead places at a time, so
// that rising paths (path[i] >= i) need no other room: a place is read before it or a later turn writes it.
// Latency bounds it: the path, the table, the values and the stores, each of a turn's places at once (256 paths of up
// to 8 tokens of 8 heads of 128 E4M3 codes, 2 MB moved: 6.6 us; one place after the other 12.5).
constexpr int kKeepAhead = 8;
__device__ const uint4 kNothing[1] = {};     // what places that are left as they are read
template <typename T, typename P>
__device__ __forceinline__ void keep_piece(const KeepArgs& a, int b, int ctx, int n, T* base, int64_t page,
                                           int64_t token) {
  const int mask = (1 << a.c.shift) - 1;
  const int* path = a.path + b * a.path_stride;
  const int* table = a.b.table + b * a.b.stride;
  for (int i0 = 0; i0 < a.path_width; i0 += kKeepAhead) {
    // no branches: the places' entries of the path, then their pages, then their values are all asked for at once
    int from[kKeepAhead], page_from[kKeepAhead], page_to[kKeepAhead];
    P v[kKeepAhead];
    bool there[kKeepAhead];
#pragma unroll
    for (int i = 0; i < kKeepAhead; i++) from[i] = path[min(i0 + i, a.path_width - 1)];
#pragma unroll
    for (int i = 0; i < kKeepAhead; i++) {
      const int slot = ctx + max(from[i], 0), to = ctx + i0 + i;
      there[i] = i0 + i < a.path_width && from[i] >= 0 && from[i] < n && from[i] != i0 + i && i0 + i < n &&
                 slot >> a.c.shift < a.b.width && to >> a.c.shift < a.b.width;
      page_from[i] = table[there[i] ? slot >> a.c.shift : 0];
      page_to[i] = table[there[i] ? to >> a.c.shift : 0];
    }
#pragma unroll
    for (int i = 0; i < kKeepAhead; i++) {
      const int id = as_page(a.c, page_from[i]);
      there[i] = there[i] && id >= 0 && as_page(a.c, page_to[i]) >= 0;
      const uint64_t src = reinterpret_cast<uint64_t>(base + id * page + ((ctx + from[i]) & mask) * token);
      v[i] = *(const __attribute__((address_space(1))) P*)(there[i] ? src : reinterpret_cast<uint64_t>(kNothing));
    }
    // one wait for all values (behind the branches' joins the compiler would let each store wait for the last one)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(7 << 4);      // vmcnt(0) expcnt(7) lgkmcnt(0)
#pragma unroll
    for (int i = 0; i < kKeepAhead; i++)
      if (there[i]) *reinterpret_cast<P*>(base + page_to[i] * page + ((ctx + i0 + i) & mask) * token) = v[i];
  }
}

__global__ void __launch_bounds__(256) k_keep(KeepArgs a, int pieces, int per) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int b = (int)(i / per);
  if (b >= a.b.n || a.b.width == 0) return;
  int u = (int)(i - (int64_t)b * per);       // [k, v][heads][pieces of 16 bytes], then [k, v][heads] scales
  const int ctx = context_of(a.b, b);
  const int n = start_of(a.b, b + 1, kMaxContext) - start_of(a.b, b, kMaxContext);
  const int all = 2 * a.c.heads * pieces;
  if (u < all) {
    const int tensor = u / (a.c.heads * pieces), h = u / pieces % a.c.heads, p = u % pieces;
    const int each = a.c.type == T_F16 || a.c.type == T_BF16 ? 8 : 16;   // elements a piece; strides are its multiples
    uint4* base = static_cast<uint4*>(tensor ? a.c.v : a.c.k) + h * (a.c.head / each) + p;
    keep_piece<uint4, u32x4_t>(a, b, ctx, n, base, a.c.page / each, a.c.token / each);
  } else {
    u -= all;
    const int tensor = u / a.c.heads, h = u % a.c.heads;
    keep_piece<float, float>(a, b, ctx, n, (tensor ? a.c.vs : a.c.ks) + h * a.c.shead, a.c.spage, a.c.stoken);
  }
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, hipStream_t s) {
  const RopeArgs& r = a.r;
  const int64_t tokens = r.tokens;
  const bool bf = r.type == T_BF16;
  if (!wide(a)) {
    const int64_t units = tokens * (r.op[0].heads + 2 * a.c.heads);
    if (!launchable((units + 3) / 4, 256)) return hipErrorInvalidConfiguration;
    const auto k = bf ? k_append_any<true> : k_append_any<false>;
    hipLaunchKernelGGL(k, dim3((unsigned)((units + 3) / 4)), dim3(256), 0, s, a, units);
    return hipGetLastError();
  }
  int lanes = 1;
  while (lanes * 16 < r.dim) lanes *= 2;
  const int groups = 64 / lanes;
  constexpr int U = 2;
  const int per = U * groups;
  Splits sp{};
  int64_t blocks = 0;
  for (int i = 0; i < 2; i++) {
    Split& w = sp.of[i];
    w.heads = i ? 2 * a.c.heads : r.op[0].heads;
    if (!w.heads) continue;                  // no queries
    w.batches = (w.heads + per - 1) / per;
    // all heads of several tokens where they fit a wave and the table, with two waves left per SIMD
    int64_t tw = per / w.heads < 1024 / r.dim ? per / w.heads : 1024 / r.dim;
    tw = tw < tokens / 2048 ? tw : tokens / 2048;
    w.tw = tw < 1 ? 1 : (int)tw;
    const int64_t waves = (tokens + w.tw - 1) / w.tw * w.batches;
    if (waves >= (int64_t)1 << 28) return hipErrorInvalidConfiguration;
    w.waves = (int)waves;
    blocks += (waves + 3) / 4;
  }
  if (!launchable(blocks, 256)) return hipErrorInvalidConfiguration;
  const auto k = r.halves && 2 * r.pairs < r.dim ? (bf ? k_append<true, HALVES_PARTIAL, U> : k_append<false, HALVES_PARTIAL, U>)
                 : r.halves              ? (bf ? k_append<true, HALVES, U> : k_append<false, HALVES, U>)
                 : 2 * r.pairs < r.dim ? (bf ? k_append<true, PARTIAL, U> : k_append<false, PARTIAL, U>)
                                       : (bf ? k_append<true, ADJACENT, U> : k_append<false, ADJACENT, U>);
  hipLaunchKernelGGL(k, dim3((unsigned)blocks), dim3(256), 0, s, a, lanes, sp);
  return hipGetLastError();
}

hipError_t launch_keep(const KeepArgs& a, hipStream_t s) {
  const bool half = a.c.type == T_F16 || a.c.type == T_BF16;
  const int pieces = half ? a.c.dim / 8 : a.c.dim / 16;
  const int64_t per = (int64_t)2 * a.c.heads * (pieces + (half ? 0 : 1));
  const int64_t blocks = (per * a.b.n + 255) / 256;
  if (!launchable(blocks, 256) || per >= (int64_t)1 << 31) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(k_keep, dim3((unsigned)blocks), dim3(256), 0, s, a, pieces, (int)per);
  return hipGetLastError();
}

}  // namespace svdq
