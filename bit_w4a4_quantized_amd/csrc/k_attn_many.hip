// Attention of a step's tokens over a paged cache (svdq_tree_attention), for many rows a cache head: large trees
// and chunks of prompts.  The mathematics is k_attn_few's; here the matrix cores bound it
// (with the exponentials: a chunk of 4096 over 12288 bf16 keys of 24 heads of 128, 722 GFLOP: 730 to 790 us, 915 to
// 990 TFLOP/s, matrix cores busy for half of it; over an E4M3 cache 990 to 1030), and the loads of few keys' tiles.
//
// A workgroup has 128 rows of one sequence and cache head (and a part of the keys), each of its four waves 32 of
// them; all four share tiles of 64 keys (32 of heads past 128), which come to LDS by loads of their own while the tile before is in work
// (codes of an 8-bit cache through registers, where they become fp16).  As in k_attn_few the products are
// transposed, S^T = K Q^T and O^T = V^T P^T, here 32 x 32 a result: lane l has half of the probabilities of row
// l % 32, keys 8 (i / 4) + 4 (l / 32) + i % 4 of each 32, and feeds them to the second product as they are.
//
// Pieces of 16 bytes are stored turned by the row's number, so that neither the first product's reads (one piece
// of 32 rows) nor the second's transposed ones (64 bytes of four rows) meet in a bank.
#include "paged_attn.h"

namespace svdq {

namespace {

using namespace attn;

// Where the piece p of a row lies in its row.
template <int DP>
__device__ __forceinline__ int turn_k(int row) { return DP == 64 ? (row >> 1) & 7 : DP == 128 ? row & 15 : row & 7; }
template <int DP>
__device__ __forceinline__ int turn_v(int row) { return DP == 64 ? (row >> 1 & 1) << 2 : (row & 3) << 2; }

constexpr float kFar = 0x1p20f;              // logits (in powers of two) from here on have steps of an eighth and more

__device__ const uint4 kNothing[1] = {};     // 16 bytes of zeros that loads of absent keys read

__device__ __forceinline__ uint64_t same_in_wave(uint64_t x) {
  return ((uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(x >> 32)) << 32) | (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)x);
}

// Lane l's 16 bytes at `from` to LDS at `to` + 16 l; `to` is the wave's.  Written out, because the compiler cannot
// tell which of the two tiles a transposed read takes and would wait for the other's loads in front of it.  It has no
// results in registers; ready() below waits for it.  Nothing else here keeps a value in m0.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void to_lds(uint64_t from, uint16_t* to) {
  const uint32_t at = (uint32_t)(uintptr_t)(lds_void*)to;
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(at) : "memory", "m0");
}
__device__ __forceinline__ void to_lds(uint64_t base, uint32_t off, uint32_t at) {       // base: the wave's
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(at) : "memory", "m0");
}
#pragma clang diagnostic pop

template <bool BF>
__device__ __forceinline__ v16f mfma32(const v4u& x, const v4u& y, const v16f& z) {
  if (BF) return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, x), __builtin_bit_cast(v8bf, y), z, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, x), __builtin_bit_cast(v8h, y), z, 0, 0, 0);
}

template <bool BF, int CK, int DP>
__global__ void __launch_bounds__(256, DP == 256 ? 1 : 2) k_attn_many(AttnArgs a) {
  constexpr int BN = DP == 256 ? 32 : 64;    // keys a tile: the registers of 64 do not fit beside results of 256
  constexpr int NB = BN / 32;
  constexpr uint64_t kAll = ~0ull >> (64 - BN);
  constexpr int kSteps = DP / 16;            // of the first product's contraction
  constexpr int kBlocks = DP / 32;           // results of the second
  constexpr int kAhead = 4;
  constexpr int kPieces = CK == C16 ? DP / 8 : DP / 16;   // 16-byte pieces a row of the cache
  constexpr int kRows = 64 / kPieces;        // rows that a wave's load takes
  constexpr int kLoads = BN / 4 / kRows;     // of a wave, for its share of a tile's K, or V
  __shared__ __attribute__((aligned(16))) uint16_t tiles[4 * BN * DP];     // K, V and the other tile's
  constexpr int kScales = CK == C16 ? 4 : BN + 4;
  // scales of K and V, and the latter's logarithms with the tile's largest behind them
  __shared__ __attribute__((aligned(16))) float s0[3][kScales], s1[3][kScales];
  __shared__ int sick;                       // some tile of V held an infinity or NaN
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 31, half = lane >> 5;

  Work w;
  if (!cut_work<128>(a, w)) return;          // the whole workgroup
  const int begin = w.begin, end = w.end, dim = a.c.dim;

  // the lane's row and its queries
  const int r = w.row0 + 32 * wave + c;
  const bool valid = r < w.rows;
  const int tok = valid ? r / a.group : 0;
  const int wave_last = min(w.row0 + 32 * wave + 31, w.rows - 1) / a.group;      // the wave's last token, and its first
  const int wave_first = min(w.row0 + 32 * wave, w.rows - 1) / a.group;
  v4u qf[kSteps];
  {
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + (int64_t)(w.s0 + tok) * a.q_token +
                        (int64_t)(w.head * a.group + r - tok * a.group) * a.q_head;
#pragma unroll
    for (int s = 0; s < kSteps; s++) {
      const int d = s * 16 + half * 8;
      qf[s] = v4u{0, 0, 0, 0};
      if (valid && d < dim) __builtin_memcpy(&qf[s], q + d, 16);
    }
  }
  float coef = a.scale;
  if (CK != C16) coef = power_of_two(scale_power(a) + (a.qbf ? queries_to_f16<kSteps, 32>(qf) : 0));

  v16f acc[kBlocks];
#pragma unroll
  for (int d = 0; d < kBlocks; d++)
#pragma unroll
    for (int i = 0; i < 16; i++) acc[d][i] = 0.f;
  float m = -INFINITY, l = 0.f, r_v = 0.f;
  bool far_rows = false;                     // some row of the wave has its reference at kFar or beyond (16-bit caches)

  constexpr int es = CK == C16 ? 2 : 1;
  const uint8_t* kbase = static_cast<const uint8_t*>(a.c.k) + w.head * a.c.head * es;
  const uint8_t* vbase = static_cast<const uint8_t*>(a.c.v) + w.head * a.c.head * es;

  // addresses as numbers: chosen without a branch
  const uint64_t kaddr = reinterpret_cast<uint64_t>(kbase), vaddr = reinterpret_cast<uint64_t>(vbase);
  const uint64_t nothing = reinterpret_cast<uint64_t>(kNothing);
  // A load's rows are first_row(i) + lane / kPieces.  Their turns do not depend on i, so that where one page holds a
  // load's rows the lane's place behind the first of them is the same for all loads and tiles.  (Strides past
  // 32 bits, and pages of fewer rows, go the slow way.)
  auto first_row = [&](int i) { return (i * 4 + wave) * kRows; };
  const int row_in = lane / kPieces, piece = lane % kPieces;
  const int pk = CK == C16 ? piece ^ turn_k<DP>(first_row(0) + row_in) : piece;
  const int pv = CK == C16 ? piece ^ turn_v<DP>(first_row(0) + row_in) : piece;
  const bool in_k = pk * (16 / es) < dim, in_v = pv * (16 / es) < dim;     // not past the head's end
  const uint32_t page_bytes = (uint32_t)(a.c.page * es), token_bytes = (uint32_t)(a.c.token * es);
  const uint32_t kat = row_in * token_bytes + pk * 16, vat = row_in * token_bytes + pv * 16;
  const int page_size = 1 << a.c.shift, page_mask = page_size - 1;
  const bool steady = page_size >= kRows && a.c.page < (int64_t)1 << 31 && a.c.token < 1 << 24;
  if (dim < DP) {                            // places past the head's end are never loaded: zeros for good
    for (int i = threadIdx.x; i < 4 * BN * DP / 8; i += 256) *reinterpret_cast<v4u*>(tiles + i * 8) = v4u{0, 0, 0, 0};
    __syncthreads();
  }

  v4u kr[CK == C16 ? 1 : kLoads], vr[CK == C16 ? 1 : kLoads];      // codes on their way
  float ksr = 0.f, vsr = 0.f;
  // The page of the lane's key of a tile, asked for a tile ahead.  (By the vector unit: the scalar one's loads would be
  // waited for with the reads of LDS.)
  const int* table = a.b.table + w.seq * a.b.stride;
  int own = -1;
  auto look = [&](int base) {
    if (steady && base + BN <= end) own = table[(base + (lane & (BN - 1))) >> a.c.shift];
  };
  auto fetch_scales = [&](int base, int page) {      // of the lane's key
    if (CK != C16 && wave == 0) {
      ksr = vsr = 0.f;
      if (lane < BN && page >= 0) {
        const int64_t so = page * a.c.spage + (int64_t)((base + lane) & page_mask) * a.c.stoken + w.head * a.c.shead;
        ksr = a.c.ks[so];
        vsr = a.c.vs[so];
      }
    }
  };
  // Whether `look` has found a page for each of the tile's keys (the same in all waves), and the offsets of the first
  // rows of the wave's loads, which have one page each.
  uint64_t at[kLoads];
  auto easy = [&](int base) {
    if (!steady || base + BN > end) return false;
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      if (i > 0 && page_size >= BN) {
        at[i] = at[i - 1] + (uint64_t)4 * kRows * token_bytes;
      } else {
        const uint32_t id = (uint32_t)__builtin_amdgcn_readlane(own, first_row(i));
        at[i] = (uint64_t)id * page_bytes + (uint64_t)(uint32_t)((base + first_row(i)) & page_mask) * token_bytes;
      }
    }
    return __ballot((uint32_t)own < (uint32_t)a.c.pages) == ~0ull;
  };
  const uint32_t wave_lds = (uint32_t)(uintptr_t)(lds_void*)(tiles + first_row(0) * DP);
  auto load_k = [&](int i, int off) { to_lds(same_in_wave(kaddr + at[i]), kat, wave_lds + (off + i * 4 * kRows * DP) * 2); };
  auto load_v = [&](int i, int off) { to_lds(same_in_wave(vaddr + at[i]), vat, wave_lds + (off + i * 4 * kRows * DP) * 2); };
  // Loads a tile; which of its keys there are.
  auto fetch = [&](int base, bool is_easy, int k_off, int v_off) -> uint64_t {
    if (is_easy) {
      if (CK == C16) {
        if (in_k) {
#pragma unroll
          for (int i = 0; i < kLoads; i++) load_k(i, k_off);
        }
        if (in_v) {
#pragma unroll
          for (int i = 0; i < kLoads; i++) load_v(i, v_off);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kLoads; i++) {
          kr[i] = vr[i] = v4u{0, 0, 0, 0};
          if (in_k) {
            kr[i] = *reinterpret_cast<const v4u*>(kbase + at[i] + kat);
            vr[i] = *reinterpret_cast<const v4u*>(vbase + at[i] + vat);
          }
        }
        fetch_scales(base, own);
      }
      return kAll;
    }
    uint16_t *kt = tiles + k_off, *vt = tiles + v_off;
    // the lane's own key (base + lane) says where its row is; the others' come by exchange
    const int key = base + lane, page = lane < BN && key < end ? page_of(a.b, a.c, w.seq, key) : -1;
    const int64_t off = page < 0 ? -1 : (page * a.c.page + (int64_t)(key & page_mask) * a.c.token) * es;
    const int lo = (int)off, hi = (int)(off >> 32);
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      const int row = first_row(i) + row_in;
      const int64_t o = ((int64_t)__shfl(hi, row) << 32) | (uint32_t)__shfl(lo, row);
      if (CK == C16) {
        if (in_k) to_lds(o >= 0 ? kaddr + o + pk * 16 : nothing, kt + first_row(i) * DP);
        if (in_v) to_lds(o >= 0 ? vaddr + o + pv * 16 : nothing, vt + first_row(i) * DP);
      } else {
        kr[i] = vr[i] = v4u{0, 0, 0, 0};
        if (o >= 0 && in_k) {
          kr[i] = *reinterpret_cast<const v4u*>(kbase + o + piece * 16);
          vr[i] = *reinterpret_cast<const v4u*>(vbase + o + piece * 16);
        }
      }
    }
    fetch_scales(base, page);
    return __ballot(page >= 0);
  };
  auto settle = [&](uint16_t* kt, uint16_t* vt, float (*sc)[kScales]) {      // codes to LDS
    if (CK == C16) return;
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      const int row = first_row(i) + row_in, p = 2 * piece;
#pragma unroll
      for (int x = 0; x < 2; x++) {
        *reinterpret_cast<v4u*>(kt + row * DP + ((p + x) ^ turn_k<DP>(row)) * 8) = widen<CK>(kr[i], x);
        // odd rows the other way round: two rows' pieces then reach every bank (34 x 30 over 2981 E4M3 185 -> 175 us)
        const int y = x ^ (row & 1);
        *reinterpret_cast<v4u*>(vt + row * DP + ((p + y) ^ turn_v<DP>(row)) * 8) = widen<CK>(vr[i], y);
      }
    }
    if (wave == 0) {
      const float power = __builtin_amdgcn_logf(__builtin_fabsf(vsr)), most = wave_max(power);      // (of zero past BN)
      if (lane < BN) {
        sc[0][lane] = ksr * scale_factor(a);
        sc[1][lane] = vsr;
        sc[2][lane] = power;
      }
      if (lane == 0) sc[2][BN] = most;
    }
  };
  // Tiles that some row does not see whole: V without infinities and NaN (rows that see one get it at the end).
  auto clean = [&](uint16_t* vt, float (*sc)[kScales]) {
    bool found = false;
    if (CK != CI8) {
      constexpr int kMine = BN * DP / 8 / 256;
      v4u x[kMine];
#pragma unroll
      for (int i = 0; i < kMine; i++) x[i] = *reinterpret_cast<const v4u*>(vt + (threadIdx.x + 256 * i) * 8);
#pragma unroll
      for (int i = 0; i < kMine; i++)
        if (make_finite<BF>(x[i])) {
          *reinterpret_cast<v4u*>(vt + (threadIdx.x + 256 * i) * 8) = x[i];
          found = true;
        }
    }
    if (CK != C16 && threadIdx.x < BN && !(__builtin_fabsf(sc[1][CK == C16 ? 0 : threadIdx.x]) < INFINITY)) {
      sc[1][CK == C16 ? 0 : threadIdx.x] = 0.f;
      sc[2][CK == C16 ? 0 : threadIdx.x] = -INFINITY;
      found = true;
    }
    if (found) sick = 1;
    __syncthreads();
  };
  // The lane's places in a tile: the first product's piece of row c in each step (32 rows on the same turn), and the
  // second's rows of V, 4 * half + (lane % 16) / 4 and so on (every 4 rows the same).
  int kof[kSteps], vof[kBlocks];
#pragma unroll
  for (int s = 0; s < kSteps; s++) kof[s] = c * DP + ((2 * s + half) ^ turn_k<DP>(c)) * 8;
#pragma unroll
  for (int d = 0; d < kBlocks; d++) {
    const int row = 4 * half + ((lane & 15) >> 2), at = d * 32 + (lane >> 4 & 1) * 16 + (lane & 3) * 4;
    vof[d] = row * DP + ((at >> 3) ^ turn_v<DP>(row)) * 8 + (at & 7);
  }

  auto compute = [&](int base, uint64_t live, const uint16_t* kt, const uint16_t* vt, bool loads, int then,
                     const float (*sc)[kScales]) {
    v16f st[NB];
#pragma unroll
    for (int b = 0; b < NB; b++)
#pragma unroll
      for (int i = 0; i < 16; i++) st[b][i] = 0.f;
    // The order is written out (the compiler's own waits for each read in front of the product that takes it): reads
    // of K run kAhead steps ahead, the first sixteen rows of V are on their way while the powers' reference is found.
    auto read_k = [&](int s, int b) { return *reinterpret_cast<const v4u*>(kt + kof[s] + b * 32 * DP); };
    auto read_v = [&](int u, int d) {
      const uint16_t* x = vt + vof[d] + u * 16 * DP;
      return transposed(x, x + 8 * DP);
    };
    v4u vf[2][kBlocks], pf[2];
    auto first_product = [&](auto between) {
      v4u kf[kAhead][NB];
#pragma unroll
      for (int s = 0; s < kAhead; s++)
#pragma unroll
        for (int b = 0; b < NB; b++) kf[s][b] = read_k(s, b);
#pragma unroll
      for (int s = 0; s < kSteps; s++) {
#pragma unroll
        for (int b = 0; b < NB; b++) st[b] = mfma32<BF>(kf[s % kAhead][b], qf[s], st[b]);
        if (s + kAhead < kSteps) {
#pragma unroll
          for (int b = 0; b < NB; b++) kf[s % kAhead][b] = read_k(s + kAhead, b);
        }
        between(s);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    constexpr int kEach = kSteps / (2 * kLoads) > 0 ? kSteps / (2 * kLoads) : 1;
    if (CK == C16 && loads) {                // the next tile's loads go out between the products
      first_product([&](int s) {
        if (s % kEach == 0 && s / kEach < 2 * kLoads) {
          if (s / kEach % 2 == 0) load_k(s / kEach / 2, then);
          else load_v(s / kEach / 2, then + BN * DP);
        }
      });
    } else {
      first_product([](int) {});
    }
#pragma unroll
    for (int d = 0; d < kBlocks; d++) vf[0][d] = read_v(0, d);
    __builtin_amdgcn_sched_barrier(0);
    // logits in powers of two
    if (CK != C16) {
#pragma unroll
      for (int b = 0; b < NB; b++)
#pragma unroll
        for (int g = 0; g < 4; g++) {
          const v4f x = *reinterpret_cast<const v4f*>(&sc[0][32 * b + 8 * g + 4 * half]);
#pragma unroll
          for (int i = 0; i < 4; i++) st[b][4 * g + i] *= x[i];
        }
    }
    const int sure = a.tree ? w.ctx : w.ctx + wave_first + 1;      // keys below it are seen by all of the wave's rows
    if (base + BN > sure || live != kAll) {  // the same in every lane
      uint32_t seen = 0;
#pragma unroll
      for (int g = 0; g < 4 * NB; g++) {
        const int k = 8 * g + 4 * half;
        seen |= (w.sees4(a, tok, base + k) & (uint32_t)(live >> k)) << (4 * g);
      }
#pragma unroll
      for (int e = 0; e < 16 * NB; e++) st[e >> 4][e & 15] = seen >> e & 1 ? st[e >> 4][e & 15] : -INFINITY;
    }
    // the references (move_powers)
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < 16 * NB; e++) top = fmaxf(top, st[e >> 4][e & 15]);
    top *= coef;
    constexpr bool kLands = CK == C16 && !BF;
    bool move = top - m > (kLands ? kLand : 0.f) + kSlack, far = false;
    if (CK != C16) move = move || ((top - m) + sc[2][CK == C16 ? 0 : BN]) - r_v > kLand + kSlack;      // a bound of the products
    if (__any(move) || far_rows) {
      // rounded as the bound is, which the products then never pass
#pragma clang fp contract(off)
      top = fmaxf(top, __shfl_xor(top, 32));
      const float old = m, sum_by = move_powers<kLands>(top, m);
      float by = sum_by;
      if (CK != C16) {
        float vtop = -INFINITY;
#pragma unroll
        for (int b = 0; b < NB; b++)
#pragma unroll
          for (int g = 0; g < 4; g++) {
            const v4f x = *reinterpret_cast<const v4f*>(&sc[2][CK == C16 ? 0 : 32 * b + 8 * g + 4 * half]);
#pragma unroll
            for (int i = 0; i < 4; i++) vtop = fmaxf(vtop, (st[b][4 * g + i] * coef - m) + x[i]);
            asm volatile("" ::: "memory");   // few at once
          }
        vtop = fmaxf(vtop, __shfl_xor(vtop, 32));
        by = move_products(vtop, m == old ? 0.f : m - old, r_v);
      }
      l *= sum_by;
#pragma unroll
      for (int d = 0; d < kBlocks; d++) acc[d] *= by;
      // The powers below take a logit's product and m in one rounding, m the rounded product of the largest: apart by up
      // to half a step of it, which must stay small.  (Products with a power of two are not rounded.)
      if (CK == C16) {
        far = __builtin_fabsf(m) >= kFar && m > -INFINITY;
        far_rows = __any(far);
        if (far) {
          // (1 / coef may lie below the normal numbers)
          const float back = __builtin_ldexpf(__builtin_amdgcn_rcpf(__builtin_ldexpf(coef, -64)), -64);
#pragma unroll
          for (int e = 0; e < 16 * NB; e++) st[e >> 4][e & 15] = (st[e >> 4][e & 15] * coef - m) * back;
        }
      }
    }
    const float mu = m == -INFINITY || far ? 0.f : m;
    const float scale_by = CK == C16 ? 1.f : __builtin_amdgcn_exp2f(-r_v);
    float part[4] = {0.f, 0.f, 0.f, 0.f};
    v4f sv[2];                               // scales of V of the lane's half of sixteen keys, read ahead of their powers
    auto read_scales = [&](int u) {
      if (CK == C16) return;
#pragma unroll
      for (int x = 0; x < 2; x++) sv[x] = *reinterpret_cast<const v4f*>(&sc[1][CK == C16 ? 0 : (2 * u + x) * 8 + 4 * half]);
    };
    // Two of sixteen keys' powers: rounded to 16 bits, with V's scales relative to 2^(m + r), as in k_attn_few.
    auto power = [&](int u, int x) {
      const int e = 8 * u + 2 * x;
      const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(st[e >> 4][e & 15], coef, -mu));
      const float q = __builtin_amdgcn_exp2f(__builtin_fmaf(st[e >> 4][(e & 15) + 1], coef, -mu));
      part[x] += p + q;
      pf[u & 1][x] = CK == C16 ? pack16(p, q, BF) : pack_f16(p * (sv[x >> 1][2 * (x & 1)] * scale_by), q * (sv[x >> 1][2 * (x & 1) + 1] * scale_by));
    };
    read_scales(0);
#pragma unroll
    for (int x = 0; x < 4; x++) power(0, x);
    // the next sixteen keys' powers and rows of V between the products of these
#pragma unroll
    for (int u = 0; u < 2 * NB; u++) {
      if (u + 1 < 2 * NB) {
        read_scales(u + 1);
#pragma unroll
        for (int d = 0; d < kBlocks; d++) vf[(u + 1) & 1][d] = read_v(u + 1, d);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int d = 0; d < kBlocks; d++) {
        acc[d] = mfma32<BF>(vf[u & 1][d], pf[u & 1], acc[d]);
        if (u + 1 < 2 * NB) {
#pragma unroll
          for (int x = 4 * d / kBlocks; x < 4 * (d + 1) / kBlocks; x++) power(u + 1, x);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    l += (part[0] + part[1]) + (part[2] + part[3]);
  };

  // ring of two tiles
  auto ready = [&]() {
    __builtin_amdgcn_s_waitcnt((7 << 4));    // vmcnt(0) expcnt(7) lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // keys below it are seen by all of the workgroup's rows
  const int all_see = a.tree ? w.ctx : w.ctx + w.row0 / a.group + 1;
  if (threadIdx.x == 0) sick = 0;            // before the first tile's barrier
  if (begin < end) {
    constexpr int kTile = BN * DP;
    look(begin);
    uint64_t live = fetch(begin, easy(begin), 0, kTile);
    look(begin + BN);
    auto turn = [&](int base, int now, int then, auto* st) {     // places of this tile and of the next
      uint16_t *kt = tiles + now, *vt = tiles + now + kTile;
      settle(kt, vt, st);
      ready();
      const bool more = base + BN < end, next_easy = more && easy(base + BN);
      // a wave whose rows see none of the tile has nothing to do (a chunk's later keys)
      const bool works = a.tree || base <= w.ctx + wave_last, checks = base + BN > all_see;
      const bool loads = CK == C16 && dim == DP && next_easy && works && !checks;
      uint64_t next = kAll;
      if (more && !loads) next = fetch(base + BN, next_easy, then, then + kTile);
      if (checks) clean(vt, st);             // the same in every wave
      if (more) look(base + 2 * BN);
      if (works) compute(base, live, kt, vt, loads, then, st);
      live = next;
    };
    for (int base = begin; base < end; base += 2 * BN) {
      turn(base, 0, 2 * kTile, s0);
      if (base + BN < end) turn(base + BN, 2 * kTile, 0, s1);
    }
  }

  l += __shfl_xor(l, 32);
  const float unit = CK == C16 ? 1.f : __builtin_amdgcn_exp2f(r_v);
  if (begin < end) {
    __syncthreads();
    if (sick) {                              // rare: key by key, each row those that it sees
#pragma unroll 1
      for (int key = max(begin, all_see / BN * BN); key < end; key++) {
        const int page = page_of(a.b, a.c, w.seq, key);
        if (page < 0) continue;
        const bool sees = valid && w.sees(a, tok, key);
#pragma unroll
        for (int d = 0; d < kBlocks; d++) {
#pragma unroll
          for (int i = 0; i < 16; i++) {
            const int at = d * 32 + 8 * (i >> 2) + 4 * half + (i & 3);
            const float x = infinite_value<BF, CK>(a, w, page, key, min(at, dim - 1));
            acc[d][i] += sees ? x : 0.f;
          }
          asm volatile("" ::: "memory");     // few loads at once
        }
      }
    }
  }
  if (!valid) return;
  const Dest to = dest_of<128>(a, w, 32 * wave + c);
#pragma unroll
  for (int d = 0; d < kBlocks; d++)
#pragma unroll
    for (int g = 0; g < 4; g++) {
      const int at = d * 32 + 8 * g + 4 * half;
      if (at < dim)
        put(to, a.qbf, at, v4f{acc[d][4 * g], acc[d][4 * g + 1], acc[d][4 * g + 2], acc[d][4 * g + 3]} * unit, m, l);
    }
}

template <bool BF, int CK, int DP>
hipError_t launch(const AttnArgs& a, hipStream_t s) {
  const int64_t blocks = blocks_of(a);
  if (!launchable(blocks, 256)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_attn_many<BF, CK, DP>), dim3((unsigned)blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <bool BF, int CK>
hipError_t launch_dim(const AttnArgs& a, hipStream_t s) {
  return a.c.dim <= 64 ? launch<BF, CK, 64>(a, s) : a.c.dim <= 128 ? launch<BF, CK, 128>(a, s) : launch<BF, CK, 256>(a, s);
}

}  // namespace

hipError_t attn::launch_many(const AttnArgs& a, hipStream_t s) {
  switch (a.c.type) {
    case T_F16: return launch_dim<false, C16>(a, s);
    case T_BF16: return launch_dim<true, C16>(a, s);
    case T_INT8: return launch_dim<false, CI8>(a, s);
    default: return launch_dim<false, CE4>(a, s);
  }
}

}  // namespace svdq
