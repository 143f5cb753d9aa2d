// Attention of a step's tokens over a paged cache (svdq_tree_attention), for few rows a cache head:
//
//   o[t, h] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q[t, h] . k_j - m)
//
// over the keys j of the token's sequence that it sees: the context's, and of the step's own tokens those
// that its row of the tree marks (or, without a tree, those up to itself).  One pass over the keys with the
// running maximum and sum of the softmax.
//
// The cache's bytes bound it (64 sequences over up to 8000 int8 keys of 8 heads of 128, 812 MB: 168 us, 4.8 TB/s, the
// rate of a large copy; one over 131072 E4M3 keys, 277 MB: 64 us), the loads' latency where it is short (1000 bf16 keys:
// 8.4 us).  A row is a token and one of the `group` query heads that share a cache head;
// a workgroup has 16 NT rows of one sequence and cache head and a part of the keys, its waves take turns at
// tiles of 32 keys, each with sums of its own, joined at the end through LDS and over the parts by
// k_attn_join.  Nothing is shared between the waves in between, so there is no barrier in the loop and the
// loads of many waves are in flight at once.
//
// Per tile the transposed products keep a row's values in one lane column: S^T = K Q^T (16 keys a result
// tile) and O^T = V^T P^T.  A lane then has 8 of the 32 probabilities of its row c = lane % 16, in just the
// order in which it feeds them back as the second product's operand: keys 16 t + 4 (lane / 16) + i in place
// 4 t + i of the contraction, and V is read from LDS in that order, transposed on the way.
#include "paged_attn.h"

namespace svdq {

namespace {

using namespace attn;

// Waves a SIMD that the registers are kept to.
constexpr int few_waves(int CK, int DP, int NT) { return DP == 256 ? 1 : DP == 64 ? 3 : NT == 2 || CK == C16 ? 2 : 3; }

template <int CK, int DP, int NT, int NW>
struct FewLds {
  // V's rows of 2 DP bytes and 32 more: eight of them side by side reach every bank
  __attribute__((aligned(16))) uint16_t v[NW][32 * (DP + 16)];
  __attribute__((aligned(16))) float s[CK == C16 ? 1 : NW][2][32];   // scales of K and V
  float ml[NW][16 * NT][2];
};

template <bool BF, int CK, int DP, int NT, int NW>
__device__ __forceinline__ void attend(const AttnArgs& a, const Work& w, FewLds<CK, DP, NT, NW>& lds) {
  constexpr int kV = DP + 16;                // halves a row of V in LDS
  constexpr int kSteps = DP / 32;            // of the contraction over the head's values
  constexpr int kPieces = CK == C16 ? DP / 8 : DP / 16;   // 16-byte pieces a row of the cache
  constexpr int kLoads = kPieces / 2;        // of a lane, for 32 rows of V
  constexpr int kRows = 64 / kPieces;        // of V a load instruction
  auto& lds_v = lds.v;
  auto& lds_s = lds.s;
  auto& lds_ml = lds.ml;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, c = lane & 15, quad = lane >> 4;

  const int begin = w.begin, end = w.end, dim = a.c.dim;

  // rows and their queries
  int tok[NT];
  bool valid[NT];
  float coef[NT];
  v4u qf[NT][kSteps];
#pragma unroll
  for (int n = 0; n < NT; n++) {
    const int r = w.row0 + 16 * n + c;
    valid[n] = r < w.rows;
    const int i = r / a.group;
    tok[n] = valid[n] ? i : 0;
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + (int64_t)(w.s0 + tok[n]) * a.q_token +
                        (int64_t)(w.head * a.group + r - i * a.group) * a.q_head;
#pragma unroll
    for (int s = 0; s < kSteps; s++) {
      const int d = CK == C16 ? s * 32 + quad * 8 : (s >> 1) * 64 + quad * 16 + (s & 1) * 8;
      qf[n][s] = v4u{0, 0, 0, 0};
      if (valid[n] && d < dim) __builtin_memcpy(&qf[n][s], q + d, 16);
    }
    coef[n] = a.scale;
    if (CK != C16) coef[n] = power_of_two(scale_power(a) + (a.qbf ? queries_to_f16<kSteps, 16>(qf[n]) : 0));
  }

  v4f acc[NT][DP / 16];
  bool sick = false;                         // the lane has taken an infinity or NaN out of V
  float m[NT], l[NT], r[NT];
#pragma unroll
  for (int n = 0; n < NT; n++) {
    m[n] = -INFINITY;
    l[n] = r[n] = 0.f;
#pragma unroll
    for (int dt = 0; dt < DP / 16; dt++) acc[n][dt] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  uint16_t* vt = lds_v[wave];
  constexpr int es = CK == C16 ? 2 : 1;
  constexpr int kKLoads = CK == C16 ? kSteps : kSteps / 2;         // pieces of a row of K that a lane takes
  const uint8_t* kbase = static_cast<const uint8_t*>(a.c.k) + w.head * a.c.head * es;
  const uint8_t* vbase = static_cast<const uint8_t*>(a.c.v) + w.head * a.c.head * es;
  const int l32 = lane & 31, page_mask = (1 << a.c.shift) - 1;

  // A tile's keys in flight, K and V as whole rows (a lane's operands of K straight from memory, 64 bytes of 16 rows
  // an instruction, came at 4.4 TB/s where whole lines come at 5.4).
  v4u kr[kLoads], vr[kLoads];
  float ks = 0.f, vs = 0.f;
  uint32_t live = 0;                         // which of its keys there are
  int64_t off = 0;                           // of the row of the lane's key; with a page of its own the tile's first
  bool easy = false;                         // one page holds the tile, and all of its keys are there
  const bool steady = page_mask >= 31 && a.c.page < (int64_t)1 << 31 && a.c.token < 1 << 24;
  const uint32_t page_bytes = (uint32_t)(a.c.page * es), token_bytes = (uint32_t)(a.c.token * es);
  const int row_in = lane / kPieces, piece = lane % kPieces;
  auto entry_at = [&](int base) {            // of key base + lane % 32
    const int key = base + l32;
    return key < end ? entry_of(a.b, a.c, w.seq, key) : -1;
  };
  auto find = [&](int base, int entry) {
    const int page = as_page(a.c, entry);
    live = (uint32_t)__ballot(page >= 0);
    easy = steady && live == 0xFFFFFFFFu;
    const int64_t in_page = (base + l32) & page_mask;
    if (easy) {
      const uint32_t id = (uint32_t)__builtin_amdgcn_readfirstlane(page);
      off = (int64_t)((uint64_t)id * page_bytes + (uint64_t)(uint32_t)(base & page_mask) * token_bytes);
    } else {
      off = page < 0 ? -1 : (page * a.c.page + in_page * a.c.token) * es;
    }
    if (CK != C16) {
      ks = vs = 0.f;
      if (page >= 0) {
        const int64_t so = page * a.c.spage + in_page * a.c.stoken + w.head * a.c.shead;
        ks = a.c.ks[so];
        vs = a.c.vs[so];
      }
    }
  };
  // Places past the head's end read its first piece instead (in V they make results that nothing takes; in K they
  // are made zeros on the way to LDS, to meet those of the queries).
  const bool in = piece * (16 / es) < dim;
  const uint32_t place = row_in * token_bytes + (in ? piece * 16 : 0);
  auto load = [&](const uint8_t* from, v4u (&r)[kLoads]) {
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      if (easy) {
        r[i] = *reinterpret_cast<const v4u*>(from + off + i * kRows * token_bytes + place);
      } else {
        const int row = i * kRows + row_in;
        const int64_t o = ((int64_t)__shfl((int)(off >> 32), row) << 32) | (uint32_t)__shfl((int)off, row);
        r[i] = v4u{0, 0, 0, 0};
        if (o >= 0) r[i] = *reinterpret_cast<const v4u*>(from + o + (in ? piece * 16 : 0));
      }
    }
  };
  constexpr int kK = CK == C16 ? 2 * kV : DP + 16;       // bytes a row of K in LDS, where V comes after it
  uint8_t* kt = reinterpret_cast<uint8_t*>(vt);

  int base = begin + wave * 32, entry = entry_at(base);
  if (base < end) {
    find(base, entry);
    load(kbase, kr);
    load(vbase, vr);
    entry = entry_at(base + 32 * NW);
  }
  for (; base < end; base += 32 * NW) {
    const bool masked = base + 32 > w.ctx || live != 0xFFFFFFFFu, more = base + 32 * NW < end;   // the same in every lane
    uint32_t seen[NT];
    if (masked) {
#pragma unroll
      for (int n = 0; n < NT; n++) {
        seen[n] = 0;
#pragma unroll 1                             // (unrolled, 64 x 8000 int8 took 207 us for 169)
        for (int t = 0; t < 2; t++) {
          const int k = 16 * t + 4 * quad;
          seen[n] |= (w.sees4(a, tok[n], base + k) & (live >> k)) << (4 * t);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();         // the last tile's reads of LDS are done
    if (CK != C16 && lane < 32) {
      lds_s[wave][0][lane] = ks * scale_factor(a);
      const bool infinite = masked && !(__builtin_fabsf(vs) < INFINITY);
      lds_s[wave][1][lane] = infinite ? 0.f : vs;
      sick = sick || infinite;
    }
#pragma unroll
    for (int i = 0; i < kLoads; i++)
      *reinterpret_cast<v4u*>(kt + (i * kRows + row_in) * kK + piece * 16) = in ? kr[i] : v4u{0, 0, 0, 0};
    if (more) {                              // the next tile's loads, into registers that are free now
      find(base + 32 * NW, entry);
      load(kbase, kr);
      entry = entry_at(base + 64 * NW);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();

    // S^T
    v4f st[NT][2];
#pragma unroll
    for (int n = 0; n < NT; n++) st[n][0] = st[n][1] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
      for (int s = 0; s < kKLoads; s++) {
        const v4u x = *reinterpret_cast<const v4u*>(kt + (16 * t + c) * kK + s * 64 + quad * 16);
#pragma unroll
        for (int h = 0; h < (CK == C16 ? 1 : 2); h++) {
          const v4u kk = CK == C16 ? x : widen<CK>(x, h);
#pragma unroll
          for (int n = 0; n < NT; n++) st[n][t] = mfma16<BF>(kk, qf[n][CK == C16 ? s : 2 * s + h], st[n][t]);
        }
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      uint16_t* to = vt + (i * kRows + row_in) * kV + piece * (CK == C16 ? 8 : 16);
      v4u x[2] = {CK == C16 ? vr[i] : widen<CK>(vr[i], 0), CK == C16 ? vr[i] : widen<CK>(vr[i], 1)};
      if (masked && CK != CI8) {             // rows that see an infinity or NaN get it at the end
        sick = make_finite<BF>(x[0]) || sick;
        if (CK != C16) sick = make_finite<BF>(x[1]) || sick;
      }
      *reinterpret_cast<v4u*>(to) = x[0];
      if (CK != C16) *reinterpret_cast<v4u*>(to + 8) = x[1];
      if (CK != C16) __builtin_amdgcn_sched_barrier(0);      // few pieces as fp16 at once
    }
    if (more) load(vbase, vr);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();

    // logits in powers of two
    float z[NT][8], vsc[8];
    if (CK != C16) {
#pragma unroll
      for (int t = 0; t < 2; t++) {
        const v4f x = *reinterpret_cast<const v4f*>(&lds_s[wave][0][16 * t + 4 * quad]);
        const v4f y = *reinterpret_cast<const v4f*>(&lds_s[wave][1][16 * t + 4 * quad]);
#pragma unroll
        for (int i = 0; i < 4; i++) {
          vsc[4 * t + i] = y[i];
#pragma unroll
          for (int n = 0; n < NT; n++) z[n][4 * t + i] = st[n][t][i] * x[i] * coef[n];
        }
      }
    } else {
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int e = 0; e < 8; e++) z[n][e] = st[n][e >> 2][e & 3] * coef[n];
    }
    if (masked) {
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int e = 0; e < 8; e++) z[n][e] = seen[n] >> e & 1 ? z[n][e] : -INFINITY;
    }
    // the references (move_powers)
    constexpr bool kLands = CK == C16 && !BF;
    float top[NT], most = 0.f;               // most: a bound of the lane's products against its largest logit
    bool move = false;
    if (CK != C16) {
#pragma unroll
      for (int e = 0; e < 8; e++) most = fmaxf(most, __builtin_fabsf(vsc[e]));
      most = __builtin_amdgcn_logf(most);
    }
#pragma unroll
    for (int n = 0; n < NT; n++) {
      top[n] = -INFINITY;
#pragma unroll
      for (int e = 0; e < 8; e++) top[n] = fmaxf(top[n], z[n][e]);
      move = move || top[n] - m[n] > (kLands ? kLand : 0.f) + kSlack;
      if (CK != C16) move = move || ((top[n] - m[n]) + most) - r[n] > kLand + kSlack - 0.01f;      // less what it rounds
    }
    if (__any(move)) {
#pragma unroll
      for (int n = 0; n < NT; n++) {
        top[n] = fmaxf(top[n], __shfl_xor(top[n], 16));
        top[n] = fmaxf(top[n], __shfl_xor(top[n], 32));
        const float old = m[n], sum_by = move_powers<kLands>(top[n], m[n]);
        float by = sum_by;
        if (CK != C16) {
          float vtop = -INFINITY;
#pragma unroll
          for (int e = 0; e < 8; e++) vtop = fmaxf(vtop, (z[n][e] - m[n]) + __builtin_amdgcn_logf(__builtin_fabsf(vsc[e])));
          vtop = fmaxf(vtop, __shfl_xor(vtop, 16));
          vtop = fmaxf(vtop, __shfl_xor(vtop, 32));
          by = move_products(vtop, m[n] == old ? 0.f : m[n] - old, r[n]);
        }
        l[n] *= sum_by;
#pragma unroll
        for (int dt = 0; dt < DP / 16; dt++) acc[n][dt] *= by;
      }
    }
    v4u pf[NT];
#pragma unroll
    for (int n = 0; n < NT; n++) {
      const float mu = m[n] == -INFINITY ? 0.f : m[n], scale_by = CK == C16 ? 1.f : __builtin_amdgcn_exp2f(-r[n]);
#pragma unroll
      for (int e = 0; e < 8; e++) {
        z[n][e] = __builtin_amdgcn_exp2f(z[n][e] - mu);
        l[n] += z[n][e];
      }
      // Rounded to 16 bits for the matrix cores (the sum above is of the unrounded): half an ulp of each
      // term, or 2^-32 of the largest that the row has seen (move_powers).  With 8-bit caches V's scale joins here.
#pragma unroll
      for (int e = 0; e < 4; e++)
        pf[n][e] = CK == C16 ? pack16(z[n][2 * e], z[n][2 * e + 1], BF)
                             : pack_f16(z[n][2 * e] * (vsc[2 * e] * scale_by), z[n][2 * e + 1] * (vsc[2 * e + 1] * scale_by));
    }
#pragma unroll
    for (int dt = 0; dt < DP / 16; dt++) {
      const uint16_t* at = vt + (quad * 4 + (c >> 2)) * kV + dt * 16 + (c & 3) * 4;
      const v4u vv = transposed(at, at + 16 * kV);
#pragma unroll
      for (int n = 0; n < NT; n++) acc[n][dt] = mfma16<BF>(vv, pf[n], acc[n][dt]);
    }
  }

  if (__any(sick)) {                         // rare: the wave's keys one by one, each row those that it sees
#pragma unroll 1
    for (int key = begin; key < end; key++) {
      if ((key - begin) / 32 % NW != wave) continue;
      const int page = page_of(a.b, a.c, w.seq, key);
      if (page < 0) continue;
#pragma unroll
      for (int n = 0; n < NT; n++) {
        const bool sees = valid[n] && w.sees(a, tok[n], key);
#pragma unroll
        for (int dt = 0; dt < DP / 16; dt++) {
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const float x = infinite_value<BF, CK>(a, w, page, key, min(dt * 16 + quad * 4 + i, dim - 1));
            acc[n][dt][i] += sees ? x : 0.f;
          }
          asm volatile("" ::: "memory");     // few loads at once
        }
      }
    }
  }

  // the waves' sums joined
#pragma unroll
  for (int n = 0; n < NT; n++) {
    l[n] += __shfl_xor(l[n], 16);
    l[n] += __shfl_xor(l[n], 32);
    if (quad == 0) {
      lds_ml[wave][16 * n + c][0] = m[n];
      lds_ml[wave][16 * n + c][1] = l[n];
    }
  }
  constexpr int CH = DP / NT;                // columns a turn: NW * 16 NT rows of them take V's room
  constexpr int kP = CH / 4;                 // pieces of four
  float unit[NT];
#pragma unroll
  for (int n = 0; n < NT; n++) unit[n] = CK == C16 ? 1.f : __builtin_amdgcn_exp2f(r[n]);
#pragma unroll
  for (int turn = 0; turn < NT; turn++) {
    __syncthreads();
    float* mine = reinterpret_cast<float*>(vt);
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int x = 0; x < CH / 16; x++) {
        const v4f v = acc[n][turn * (CH / 16) + x] * unit[n];
        *reinterpret_cast<v4f*>(mine + (16 * n + c) * CH + (((x * 4 + quad) ^ c) & (kP - 1)) * 4) = v;
      }
    __syncthreads();
    for (int u = tid; u < 16 * NT * kP; u += 64 * NW) {
      const int row = u / kP, piece = u % kP, d = turn * CH + piece * 4;
      if (w.row0 + row >= w.rows || d >= dim) continue;
      float mm = -INFINITY, sum = 0.f;
      for (int x = 0; x < NW; x++) mm = fmaxf(mm, lds_ml[x][row][0]);
      v4f o{0.f, 0.f, 0.f, 0.f};
      for (int x = 0; x < NW; x++) {
        const float f = lds_ml[x][row][0] == mm ? 1.f : __builtin_amdgcn_exp2f(lds_ml[x][row][0] - mm);
        sum += f * lds_ml[x][row][1];
        const float* at = reinterpret_cast<const float*>(lds_v[x]) + row * CH + ((piece ^ (row & 15)) & (kP - 1)) * 4;
        o += f * *reinterpret_cast<const v4f*>(at);
      }
      put(dest_of<16 * NT>(a, w, row), a.qbf, d, o, mm, sum);
    }
  }
}

template <bool BF, int CK, int DP, int NT, int NW>
__global__ void __launch_bounds__(64 * NW, few_waves(CK, DP, NT)) k_attn_few(AttnArgs a) {
  __shared__ FewLds<CK, DP, NT, NW> lds;
  Work w;
  if (cut_work<16 * NT>(a, w)) attend<BF, CK, DP, NT, NW>(a, w, lds);        // the whole workgroup
}

template <bool BF, int CK, int DP, int NT>
hipError_t launch(const AttnArgs& a, hipStream_t s) {
  constexpr int NW = 4;
  const int64_t blocks = blocks_of(a);
  if (blocks > 2 * kGridRow) return hipErrorInvalidConfiguration;
  const dim3 grid = blocks < 2 * kGridRow ? dim3((unsigned)blocks) : dim3(kGridRow, 2);
  hipLaunchKernelGGL((k_attn_few<BF, CK, DP, NT, NW>), grid, dim3(64 * NW), 0, s, a);
  return hipGetLastError();
}

template <bool BF, int CK>
hipError_t launch_dim(const AttnArgs& a, hipStream_t s) {
  if (a.rows == 16)
    return a.c.dim <= 64 ? launch<BF, CK, 64, 1>(a, s) : a.c.dim <= 128 ? launch<BF, CK, 128, 1>(a, s) : launch<BF, CK, 256, 1>(a, s);
  return a.c.dim <= 64 ? launch<BF, CK, 64, 2>(a, s) : launch<BF, CK, 128, 2>(a, s);
}

}  // namespace

hipError_t attn::launch_few(const AttnArgs& a, hipStream_t s) {
  switch (a.c.type) {
    case T_F16: return launch_dim<false, C16>(a, s);
    case T_BF16: return launch_dim<true, C16>(a, s);
    case T_INT8: return launch_dim<false, CI8>(a, s);
    default: return launch_dim<false, CE4>(a, s);
  }
}

}  // namespace svdq
