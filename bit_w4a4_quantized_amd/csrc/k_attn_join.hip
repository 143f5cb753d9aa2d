// The parts of a row's keys joined: o = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s, m the largest m_s, in a fixed
// order whatever order the parts ended in.  And the choice of kernel and parts.
#include "paged_attn.h"

namespace svdq {

namespace {

using namespace attn;

// A row's values are P lanes' pieces of four; `deep` such groups share a row's parts (part s goes to group
// s % deep), joined through LDS: with few rows of many parts one group would wait for one load after another.
template <int R, int P>
__global__ void __launch_bounds__(256) k_attn_join(AttnArgs a, int deep) {
  __shared__ __attribute__((aligned(16))) float lds[256][4];
  __shared__ float lds_ml[256 / P][2];
  const int per = 256 / P / deep;            // rows a workgroup
  const int g = threadIdx.x / P, lane = threadIdx.x % P, row_in = g / deep, way = g % deep;
  const int chunks = R / per, tile = a.whole + blockIdx.x / chunks, row = (int)(blockIdx.x % chunks) * per + row_in;
  const int dim = a.c.dim, d = lane * 4;
  const int64_t id = (int64_t)(tile - a.whole) * a.parts;      // of the first part; the others follow
  const float* ml = a.part + a.ids * R * dim + (id * R + row) * 2;
  const float* o = a.part + (id * R + row) * dim + min(d, dim - 4);
  // the first parts' sums are on their way while the tile's sequence is looked up (what lies there of rows and parts that
  // a tile has not is not used)
  constexpr int kFirst = 4;
  float m4[kFirst], l4[kFirst];
  v4f o4[kFirst];
#pragma unroll
  for (int i = 0; i < kFirst; i++) {
    const int64_t s = min(way + i * deep, a.parts - 1) * (int64_t)R;
    m4[i] = ml[2 * s];
    l4[i] = ml[2 * s + 1];
    o4[i] = *reinterpret_cast<const v4f*>(o + s * dim);
  }
  Work w;
  w.id = -1;
  if (!find_tile<R>(a, tile, w)) return;     // the whole workgroup
  const Shares share = share_keys<R>(a, w, a.parts);
  // parts that have keys: the quotient to within 2^-15, up
  int parts = share.units ? (int)((float)share.units * __builtin_amdgcn_rcpf((float)share.each) + 0x1p-10f) : 0;
  parts = __builtin_amdgcn_readfirstlane(parts + (parts * share.each < share.units));
  const bool valid = w.row0 + row < w.rows && d < dim;
  float m = -INFINITY, l = 0.f;
  v4f sum{0.f, 0.f, 0.f, 0.f};
  auto add = [&](float ms, float ls, const v4f& os) {
    const float f = ms == m ? 1.f : __builtin_amdgcn_exp2f(ms - m);
    l += f * ls;
    sum += f * os;
  };
  if (valid) {
#pragma unroll
    for (int i = 0; i < kFirst; i++)
      if (way + i * deep < parts) m = fmaxf(m, m4[i]);
    for (int s = way + kFirst * deep; s < parts; s += deep) m = fmaxf(m, ml[(int64_t)s * R * 2]);
#pragma unroll
    for (int i = 0; i < kFirst; i++)
      if (way + i * deep < parts) add(m4[i], l4[i], o4[i]);
#pragma unroll 4
    for (int s = way + kFirst * deep; s < parts; s += deep) {
      const int64_t x = (int64_t)s * R;
      add(ml[2 * x], ml[2 * x + 1], *reinterpret_cast<const v4f*>(o + x * dim));
    }
  }
  if (deep > 1) {
    *reinterpret_cast<v4f*>(lds[threadIdx.x]) = sum;
    if (lane == 0) {
      lds_ml[g][0] = m;
      lds_ml[g][1] = l;
    }
    __syncthreads();
    if (way) return;
    float top = -INFINITY;
    for (int x = 0; x < deep; x++) top = fmaxf(top, lds_ml[g + x][0]);
    l = 0.f;
    sum = v4f{0.f, 0.f, 0.f, 0.f};
    for (int x = 0; x < deep; x++) {
      const float f = lds_ml[g + x][0] == top ? 1.f : __builtin_amdgcn_exp2f(lds_ml[g + x][0] - top);
      l += f * lds_ml[g + x][1];
      sum += f * *reinterpret_cast<const v4f*>(lds[threadIdx.x + x * P]);
    }
  }
  if (!valid) return;
  put(dest_of<R>(a, w, row), a.qbf, d, sum, m, l);
}

template <int R, int P>
hipError_t join(const AttnArgs& a, hipStream_t s) {
  const int64_t cuts = (int64_t)a.slots * a.c.heads - a.whole;
  // Ways: so many that each one's parts are on their way before it looks for its tile, or, where the workgroups fill
  // the chip, has eight or more (8 tiles of 16 parts: 5.7 us with 2, 3.3 with 4; 512 tiles of 6: 6.1 with 1, 8.9 with 2).
  int deep = 1;
  while (deep < 256 / P && deep * 4 <= a.parts && (deep * 8 <= a.parts || cuts * R * P * deep < 256 * 256)) deep *= 2;
  const int64_t blocks = cuts * (R / (256 / P / deep));
  if (!launchable(blocks, 256)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_attn_join<R, P>), dim3((unsigned)blocks), dim3(256), 0, s, a, deep);
  return hipGetLastError();
}

template <int R>
hipError_t join_dim(const AttnArgs& a, hipStream_t s) {
  return a.c.dim <= 64 ? join<R, 16>(a, s) : a.c.dim <= 128 ? join<R, 32>(a, s) : join<R, 64>(a, s);
}

}  // namespace

AttnPlan attn_plan(int sequences, int tokens, int heads, int kv_heads, int dim, int64_t reach, size_t room) {
  AttnPlan p{};
  const int group = heads / kv_heads;
  const int64_t each = ((int64_t)tokens * group + sequences - 1) / sequences;    // rows of a sequence and cache head
  // Past 32 rows a tile of 128 reads the cache once where tiles of 32 read it again: 16 trees of 12 over 4000 (48 rows of
  // 128 values, bf16) 80 us and 136, 64 of 9 over 2000 in E4M3 (36 rows) 125 and 125; int8 heads of 64 alone were
  // better off in tiles of 32 (56 rows over 29044: 64 us and 37), and the type is not known here.
  p.rows = each > kFewRows ? kManyRows : each > 16 && dim <= 128 ? kFewRows : 16;
  p.unit = dim > 128 && p.rows > kFewRows ? 32 : 64;
  p.slots = (int)((int64_t)tokens * group / p.rows + sequences);
  const int64_t all = (int64_t)p.slots * kv_heads;
  const int64_t tiles = (each + p.rows - 1) / p.rows * sequences * kv_heads;     // not empty, for sequences alike
  // A part has 64 keys or more, two turns of k_attn_few's four waves: a compute unit alone takes about six bytes a
  // clock from beyond its L2, so that a short context comes faster to more of them (1000 keys of 8 heads 11.2 us in
  // parts of 128, 8.6 of 64, 8.5 of 32).
  const int64_t most = reach / (p.rows <= kFewRows ? 64 : 128);
  p.whole = (int)all;
  p.parts = 1;
  const size_t id_bytes = (size_t)p.rows * (dim + 2) * sizeof(float);
  // workgroups that are on the chip at once: two a CU, three of the 16-row kernel
  const int64_t resident = p.rows == 16 ? 768 : 512;
  if (p.rows <= kFewRows) {
    // One round of workgroups, and up to four while a part is longer than its fixed costs (one sequence over 131072
    // E4M3 keys: 96 parts a head 64 + 7 us, 192 to 256 parts 62 + 12; 5 trees of 37 in 32 rows: 18.4 us for 384
    // workgroups, 18.7 for 320, 22 and more from 448 on, whose last ones wait for registers).
    const int64_t round = (p.rows == 16 ? resident : 384) / tiles;
    int64_t s = round < 1 ? 1 : round;
    while (reach / s > 1500 && s * tiles <= 2 * 768) s *= 2;
    s = s < most ? s : most;
    p.parts = s > 128 ? 128 : (int)s;
    if (p.parts > 1) p.whole = 0;
  } else {
    // The tiles of the last, partial round are cut so that it fills the chip (in rounds of whole tiles: the parts'
    // own, half a part for the workgroups that end early, and the join, whose bytes at 4.5 TB/s stand against 1.7 us
    // for 64 keys of 128 values).  Tiles that are no full round and few of many keys are cut into one round of workgroups (12
    // trees of 14 over 85055: 266 us in 16 parts, 117 in 40; 3 of 48 over 53647 in int8 137 and 38).
    //
    // Empty tiles lie evenly among the numbers: `rest` tiles with rows are in about rest * all / tiles of them.  All parts
    // together are at most three rounds of workgroups, and so are the sums that they leave (65 trees of 9 over 2000 in
    // 32 on 8 heads, 520 tiles in 664 numbers: 10 numbers cut 16 ways 152 us, none cut 145; the 152 behind the first 512 cut
    // 64 ways 261).  `reach` is the table's width, which the contexts may be far below (112 x 9 over 2000: 179 us in a
    // table for 2048 keys, 213 in one for 32768).
    const int64_t rest = tiles % resident, cut = tiles < resident ? all : (rest * all + tiles - 1) / tiles;
    const double early = tiles > resident ? 0.5 : 0.0;
    const double join = reach > 0 ? (1.1 * rest + 722.0 / dim) / reach : 0.0;
    double best = 1.0 + early;
    auto weigh = [&](int64_t s) {
      if (s > most || s > 128 || cut * s > 3 * resident) return;
      const double t = (double)((rest * s + resident - 1) / resident) / s + early / s + join * s;
      if (t < 0.95 * best) {
        best = t;
        p.parts = (int)s;
      }
    };
    if (rest) {
      for (int s = 2; s <= 16; s++) weigh(s);
      if (tiles * 16 < resident) {
        weigh(resident / 2 / rest < 128 ? resident / 2 / rest : 128);
        weigh(resident / rest < 128 ? resident / rest : 128);
      }
    }
    if (p.parts > 1) p.whole = (int)(all - cut);
  }
  if (p.parts < 2) {
    p.parts = 1;
    p.whole = (int)all;
  }
  for (;; p.parts--) {
    p.ids = (all - p.whole) * p.parts;
    p.bytes = p.parts > 1 ? p.ids * id_bytes : 0;
    if (p.bytes <= room) break;
  }
  return p;
}

hipError_t launch_attn(const AttnArgs& a, hipStream_t s) {
  const hipError_t e = a.rows <= kFewRows ? attn::launch_few(a, s) : attn::launch_many(a, s);
  if (e != hipSuccess || a.parts == 1) return e;
  return a.rows == 16 ? join_dim<16>(a, s) : a.rows == kFewRows ? join_dim<kFewRows>(a, s) : join_dim<kManyRows>(a, s);
}

}  // namespace svdq
