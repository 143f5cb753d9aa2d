// Attention of a step's tokens over a paged cache (svdq_tree_attention), for many rows a cache head: large trees
// and chunks of prompts.  The mathematics is k_attn_few's; here the matrix cores bound it.
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
__device__ __forceinline__ int turn_k(int row) { return DP == 64 ? (row >> 1) & 7 : row & 15; }
template <int DP>
__device__ __forceinline__ int turn_v(int row) { return DP == 64 ? (row >> 1 & 1) << 2 : (row & 3) << 2; }

__device__ const uint4 kNothing[1] = {};     // 16 bytes of zeros that loads of absent keys read

// Lane l's 16 bytes at `from` to LDS at `to` + 16 l; `to` is the wave's.  Written out, because the compiler cannot
// tell which of the two tiles a transposed read takes and would wait for the other's loads in front of it.  It has no
// results in registers; ready() below waits for it.  Nothing else here keeps a value in m0.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void to_lds(uint64_t from, uint16_t* to) {
  const uint32_t at = (uint32_t)(uintptr_t)(lds_void*)to;
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(at) : "memory", "m0");
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
  constexpr int kPieces = CK == C16 ? DP / 8 : DP / 16;   // 16-byte pieces a row of the cache
  constexpr int kRows = 64 / kPieces;        // rows that a wave's load takes
  constexpr int kLoads = BN / 4 / kRows;     // of a wave, for its share of a tile's K, or V
  __shared__ __attribute__((aligned(16))) uint16_t k0[BN * DP], k1[BN * DP], v0[BN * DP], v1[BN * DP];
  __shared__ __attribute__((aligned(16))) float s0[2][CK == C16 ? 4 : BN], s1[2][CK == C16 ? 4 : BN];   // scales of K and V
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 31, half = lane >> 5;

  Work w;
  if (!find_work<128>(a, w)) return;         // the whole workgroup
  const int kmax = w.last_key(a, w.row0 + 127);
  int begin, end;
  w.part(kmax, BN, &begin, &end);
  const int dim = a.c.dim;

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
  if (CK != C16 && a.qbf) coef *= queries_to_f16<kSteps, 32>(qf);

  v16f acc[kBlocks];
#pragma unroll
  for (int d = 0; d < kBlocks; d++)
#pragma unroll
    for (int i = 0; i < 16; i++) acc[d][i] = 0.f;
  float m = -INFINITY, l = 0.f, ref = 0.f;   // ref: what V's scales are taken relative to (8-bit caches)

  constexpr int es = CK == C16 ? 2 : 1;
  const uint8_t* kbase = static_cast<const uint8_t*>(a.c.k) + w.head * a.c.head * es;
  const uint8_t* vbase = static_cast<const uint8_t*>(a.c.v) + w.head * a.c.head * es;

  // addresses as numbers: chosen without a branch
  const uint64_t kaddr = reinterpret_cast<uint64_t>(kbase), vaddr = reinterpret_cast<uint64_t>(vbase);
  const uint64_t nothing = reinterpret_cast<uint64_t>(kNothing);

  // One tile: the lane's own key (base + lane) says where its row is; the others' come by exchange.
  auto entry_at = [&](int base) {
    const int key = base + lane;
    return lane < BN && key < end ? entry_of(a.b, a.c, w.seq, key) : -1;
  };
  v4u kr[CK == C16 ? 1 : kLoads], vr[CK == C16 ? 1 : kLoads];      // codes on their way
  float ksr = 0.f, vsr = 0.f;
  auto fetch = [&](int base, int page, uint16_t* kt, uint16_t* vt) {
    const int64_t in_page = (base + lane) & ((1 << a.c.shift) - 1);
    const int64_t off = page < 0 ? -1 : (page * a.c.page + in_page * a.c.token) * es;
    const int lo = (int)off, hi = (int)(off >> 32);
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      const int first = (i * 4 + wave) * kRows, row = first + lane / kPieces;
      const int64_t o = ((int64_t)__shfl(hi, row) << 32) | (uint32_t)__shfl(lo, row);
      if (CK == C16) {
        const int pk = (lane % kPieces) ^ turn_k<DP>(row), pv = (lane % kPieces) ^ turn_v<DP>(row);
        const bool there = o >= 0;
        to_lds(there && pk * 8 < dim ? kaddr + o + pk * 16 : nothing, kt + first * DP);
        to_lds(there && pv * 8 < dim ? vaddr + o + pv * 16 : nothing, vt + first * DP);
      } else {
        const int p = lane % kPieces;
        kr[i] = vr[i] = v4u{0, 0, 0, 0};
        if (o >= 0 && p * 16 < dim) {
          kr[i] = *reinterpret_cast<const v4u*>(kbase + o + p * 16);
          vr[i] = *reinterpret_cast<const v4u*>(vbase + o + p * 16);
        }
      }
    }
    if (CK != C16 && wave == 0) {
      ksr = vsr = 0.f;
      if (page >= 0) {
        const int64_t so = page * a.c.spage + in_page * a.c.stoken + w.head * a.c.shead;
        ksr = a.c.ks[so];
        vsr = a.c.vs[so];
      }
    }
  };
  auto settle = [&](uint16_t* kt, uint16_t* vt, float (*sc)[CK == C16 ? 4 : BN]) {      // codes to LDS
    if (CK == C16) return;
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      const int row = (i * 4 + wave) * kRows + lane / kPieces, p = 2 * (lane % kPieces);
#pragma unroll
      for (int x = 0; x < 2; x++) {
        *reinterpret_cast<v4u*>(kt + row * DP + ((p + x) ^ turn_k<DP>(row)) * 8) = widen<CK>(kr[i], x);
        *reinterpret_cast<v4u*>(vt + row * DP + ((p + x) ^ turn_v<DP>(row)) * 8) = widen<CK>(vr[i], x);
      }
    }
    if (wave == 0 && lane < BN) {
      sc[0][lane] = ksr;
      sc[1][lane] = vsr;
    }
  };

  auto compute = [&](int base, uint64_t live, const uint16_t* kt, const uint16_t* vt, const float (*sc)[CK == C16 ? 4 : BN]) {
    v16f st[NB];
#pragma unroll
    for (int b = 0; b < NB; b++)
#pragma unroll
      for (int i = 0; i < 16; i++) st[b][i] = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; s++)
#pragma unroll
      for (int b = 0; b < NB; b++) {
        const int row = 32 * b + c;
        const v4u kk = *reinterpret_cast<const v4u*>(kt + row * DP + ((2 * s + half) ^ turn_k<DP>(row)) * 8);
        st[b] = mfma32<BF>(kk, qf[s], st[b]);
      }
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
    const bool masked = base + BN > sure || live != kAll;          // the same in every lane
    uint32_t seen = ~0u;
    uint64_t bad = 0;
    if (masked) {
      seen = 0;
#pragma unroll 1
      for (int e = 0; e < 16 * NB; e++) {
        const int k = (e >> 2) * 8 + 4 * half + (e & 3);
        if (valid && (live >> k & 1) && w.sees(a, tok, base + k)) seen |= 1u << e;
      }
#pragma unroll
      for (int e = 0; e < 16 * NB; e++) st[e >> 4][e & 15] = seen >> e & 1 ? st[e >> 4][e & 15] : -INFINITY;
      // rows of V that hold an infinity or NaN: the product below would bring 0 * infinity to rows that do not see them
      bool sick = CK != C16 && !(__builtin_fabsf(sc[1][lane & (CK == C16 ? 3 : BN - 1)]) < INFINITY);
      if (CK != CI8)
#pragma unroll 1
        for (int p = 0; p < DP / 8; p++) sick = sick || not_finite<BF, C16>(*reinterpret_cast<const v4u*>(vt + (lane & (BN - 1)) * DP + p * 8));
      bad = __ballot(sick);
    }
    auto scale_v = [&](int e) {              // of the lane's e-th key
      const float x = sc[1][(e >> 2) * 8 + 4 * half + (e & 3)];
      return masked && !(__builtin_fabsf(x) < INFINITY) ? 0.f : x;
    };
    // the row's reference moves only when a logit passes it by kSlack (k_attn_few)
    float top = -INFINITY, vtop = 0.f;
#pragma unroll
    for (int e = 0; e < 16 * NB; e++) top = fmaxf(top, st[e >> 4][e & 15]);
    top *= coef;
    bool move = top > m + kSlack;
    if (CK != C16) {
#pragma unroll
      for (int e = 0; e < 16 * NB; e++) vtop = fmaxf(vtop, __builtin_fabsf(scale_v(e)));
      move = move || vtop > 8.f * ref;
    }
    if (__any(move)) {
      float back = 1.f;
      if (CK != C16) {
        vtop = fmaxf(vtop, ref);
        vtop = fmaxf(vtop, __shfl_xor(vtop, 32));
        back = vtop > 0.f ? ref / vtop : 1.f;
        ref = vtop;
      }
      float mn = fmaxf(top, m);
      mn = fmaxf(mn, __shfl_xor(mn, 32));
      const float f = mn == m ? 1.f : __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int d = 0; d < kBlocks; d++) acc[d] *= f * back;
    }
    const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int e = 0; e < 16 * NB; e++) {
      const float z = __builtin_amdgcn_exp2f(__builtin_fmaf(st[e >> 4][e & 15], coef, -mu));
      st[e >> 4][e & 15] = z;
      l += z;
    }
    const float inv = CK != C16 && ref > 0.f ? 1.f / ref : 0.f;
    if (bad == 0) {
      // rounded to 16 bits, with V's scales relative to ref, as in k_attn_few
#pragma unroll
      for (int u = 0; u < 2 * NB; u++) {
        v4u pf;
#pragma unroll
        for (int x = 0; x < 4; x++) {
          const int e = 8 * u + 2 * x;
          const float p = st[e >> 4][e & 15], q = st[e >> 4][(e & 15) + 1];
          pf[x] = CK == C16 ? pack16(p, q, BF) : pack_f16(p * (scale_v(e) * inv), q * (scale_v(e + 1) * inv));
        }
#pragma unroll
        for (int d = 0; d < kBlocks; d++) {
          const int row = 16 * u + 4 * half + ((lane & 15) >> 2);
          const int at = d * 32 + (lane >> 4 & 1) * 16 + (lane & 3) * 4;
          const uint16_t* x = vt + row * DP + ((at >> 3) ^ turn_v<DP>(row)) * 8 + (at & 7);
          acc[d] = mfma32<BF>(transposed(x, x + 8 * DP), pf, acc[d]);      // 8 rows on: the same turn
        }
      }
    } else {                                 // key by key, each row those that it sees
#pragma unroll 1
      for (int k = 0; k < BN; k++) {
        const int e = (k >> 3) * 4 + (k & 3), from = (k >> 2 & 1) * 32 + c;
        float p = 0.f;
#pragma unroll
        for (int x = 0; x < 16 * NB; x++)
          if (x == e) p = st[x >> 4][x & 15];
        p = __shfl(p, from);
        const bool sees = __shfl((int)(seen >> e & 1), from);
        const float vs = CK == C16 ? 1.f : sc[1][k] * inv;
#pragma unroll
        for (int d = 0; d < kBlocks; d++)
#pragma unroll
          for (int i = 0; i < 16; i++) {
            const int at = d * 32 + 8 * (i >> 2) + 4 * half + (i & 3);
            const uint32_t b = vt[k * DP + ((at >> 3) ^ turn_v<DP>(k)) * 8 + (at & 7)];
            if (sees) acc[d][i] += p * ((BF ? bf16_f32(b) : f16_f32(b)) * vs);
          }
      }
    }
  };

  // ring of two tiles
  auto ready = [&]() {
    __builtin_amdgcn_s_waitcnt((7 << 4));    // vmcnt(0) expcnt(7) lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  if (begin < end) {
    const int page = as_page(a.c, entry_at(begin));
    uint64_t live = __ballot(page >= 0);
    fetch(begin, page, k0, v0);
    int entry = entry_at(begin + BN);
    auto turn = [&](int base, uint16_t* kt, uint16_t* vt, auto* st, uint16_t* kn, uint16_t* vn) {
      settle(kt, vt, st);
      ready();
      const int page = as_page(a.c, entry);
      const uint64_t next = __ballot(page >= 0);
      if (base + BN < end) {
        fetch(base + BN, page, kn, vn);
        entry = entry_at(base + 2 * BN);
      }
      // a wave whose rows see none of the tile has nothing to do (a chunk's later keys)
      if (a.tree || base <= w.ctx + wave_last) compute(base, live, kt, vt, st);
      live = next;
    };
    for (int base = begin; base < end; base += 2 * BN) {
      turn(base, k0, v0, s0, k1, v1);
      if (base + BN < end) turn(base + BN, k1, v1, s1, k0, v0);
    }
  }

  l += __shfl_xor(l, 32);
  const float unit = CK == C16 ? 1.f : ref;
  if (!valid) return;
#pragma unroll
  for (int d = 0; d < kBlocks; d++)
#pragma unroll
    for (int g = 0; g < 4; g++) {
      const int at = d * 32 + 8 * g + 4 * half;
      if (at < dim)
        put<128>(a, w, 32 * wave + c, at, v4f{acc[d][4 * g], acc[d][4 * g + 1], acc[d][4 * g + 2], acc[d][4 * g + 3]} * unit, m, l);
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
