// svdq_gemm_act_residual on tiles (see gemm_act.h for the operator and the operands).
//
// A workgroup of WM x WN waves owns a tile of BM token rows x BN output columns, each wave TI x TJ
// MFMA tiles of 32 x 32.  K advances 128 bytes a stage through a ring of R LDS buffers filled by
// LDS-DMA: whole cache lines (64-byte row pieces fetched each line twice: 4608 x 3072 x 12288 in
// int8 214 us, 184 with the same pieces contiguous).  A stage's fragments are read half a stage
// ahead of their MFMAs, one LDS read and at most one load after each MFMA, so the matrix core works
// while the LDS serves the reads; one barrier a stage.  4608 x 3072 x 12288 takes 179 us in int8
// (1.95 PFLOP/s; 186 with GELU), 8192 cubed 2.27 PFLOP/s, in bf16 1.29, in E4M3 1.45.  The chip runs at
// 1.94 GHz under this load; neither the matrix cores (busy 45%) nor, by count, the LDS (256 KB a
// stage of a 256 x 256 tile, 2050 of its 3300 cycles at 128 bytes a cycle) are full.  Piece p (16 bytes)
// of row r sits in slot p ^ (r / 2 % 8): the reads of sixteen rows at one piece hit distinct banks.
//
// The weight tile is the MFMA's row operand: lane (r32, h) gets token row r32 and columns
// 8 q + 4 h + 0 ... 3.  The epilogue exchanges halves between the lanes of a row (two 4-column
// pieces become one of 8), applies scales, bias and activation, adds the residual and rounds;
// residual and output pass through LDS in 16 bits, so that global accesses are whole lines.
#include <math.h>

#include "gemm_act.h"

namespace svdq {
namespace gact {

namespace {

template <int TYPE>
struct Mma {
  using Acc = v16f;
};
template <>
struct Mma<T_INT8> {
  using Acc = v16i;
};
template <int TYPE>
struct Quarter {
  using Sum = v4f;
};
template <>
struct Quarter<T_INT8> {
  using Sum = v4i;
};

// A workgroup barrier after waiting for the wave's LDS operations and all but its N most recent
// vector-memory operations, with the builtins, so that the compiler's own waits know of it.
template <int N>
__device__ __forceinline__ void wait_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));   // vmcnt(N) expcnt(7) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Scheduling groups: NM MFMAs with NR LDS reads and NV vector-memory loads spread evenly after them.
template <int I, int NM, int NR, int NV>
__device__ __forceinline__ void interleave() {
  if constexpr (I < NM) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    constexpr int R0 = NR * I / NM, R1 = NR * (I + 1) / NM, V0 = NV * I / NM, V1 = NV * (I + 1) / NM;
    if constexpr (R1 > R0) __builtin_amdgcn_sched_group_barrier(0x100, R1 - R0, 0);
    if constexpr (V1 > V0) __builtin_amdgcn_sched_group_barrier(0x020, V1 - V0, 0);
    interleave<I + 1, NM, NR, NV>();
  }
}

template <int V>
struct Int {
  static constexpr int value = V;
};

template <int TYPE, int WM, int WN, int TI, int TJ, int R>
struct Tile {
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int BM = WM * 32 * TI, BN = WN * 32 * TJ;
  static constexpr int PX = BM / 8 / NW, PW = BN / 8 / NW;   // LDS-DMA instructions (8 rows each) per wave and stage
  static constexpr int BUF = (BM + BN) * BK;
  static_assert(PX * 8 * NW == BM && PW * 8 * NW == BN, "every wave moves whole 8-row pieces");
  using Acc = typename Mma<TYPE>::Acc;
  // the wave's longer side of tiles, and the other
  static constexpr bool XLONG = TI >= TJ;
  static constexpr int NO = XLONG ? TI : TJ, NI = XLONG ? TJ : TI;
  // the epilogue's staging: bytes and 16-byte slots of a wave's row, the slots a lane moves, and the
  // bits of the row that a slot is swapped by (within groups of a power of two)
  static constexpr int RB = TJ * 64, SL = TJ * 4, PASSES = TI * 32 * SL / 64, SWAP = (SL & -SL) - 1;
  static_assert(TI * 32 * SL % 64 == 0, "whole passes");
  // small tiles load the epilogue's row scales and residual before the K loop (fp16 333 x 1048 x 1999
  // with a residual 10.7 -> 9.8 us; large ones have no registers for it)
  static constexpr bool EARLY = TI * TJ == 1;
  struct Rows {
    float sx[TI];
    uint32_t res[PASSES][4];
  };
  static __device__ __forceinline__ void load_rows(const Args& a, int m0, int n0, Rows& r) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int mw = m0 + wave / WN * TI * 32, nw = n0 + wave % WN * TJ * 32;
    if (a.res) {
#pragma unroll
      for (int i = 0; i < PASSES; i++) {
        const int m = mw + (i * 64 + lane) / SL, n = nw + (i * 64 + lane) % SL * 8;
#pragma unroll
        for (int j = 0; j < 4; j++) r.res[i][j] = 0;
        if (m < a.M && n < a.N) load_piece<8>(a.res, m * a.res_stride + n, a.N - n, r.res[i]);
      }
    }
#pragma unroll
    for (int ti = 0; ti < TI; ti++) r.sx[ti] = a.xs ? a.xs[min(mw + ti * 32 + (lane & 31), a.M - 1)] : 1.f;
  }

  // The tile's product over stages first ... last - 1 of K, then the epilogue, or with `part` the
  // sums as they are to this split's place there.  cs: column scales and bias of the tile, BN
  // floats each.
  static __device__ __forceinline__ void run(const Args& a, int m0, int n0, uint8_t* b0, uint8_t* b1, uint8_t* b2,
                                             float* cs, int first, int last, Acc* part) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int h = lane >> 5, r32 = lane & 31, wm = wave / WN, wn = wave % WN;
    const int mrows = min(BM, a.M - m0), nrows = min(BN, a.N - n0);
    const rsrc_t rx = make_rsrc(a.x + (int64_t)m0 * a.x_stride, (size_t)((mrows - 1) * a.x_stride + a.KB));
    const rsrc_t rw = make_rsrc(a.w + (int64_t)n0 * a.KB, (size_t)nrows * a.KB);
    // instruction i moves rows 8 i ... 8 i + 7, lane l slot l % 8 of row 8 i + l / 8; rows past the
    // edge lie past the resource's range (the scalar offset counts) and read as zeros, like the
    // pieces past the end of K
    const int rl = lane >> 3;
    const int pe = (lane & 7) ^ (rl >> 1), po = pe ^ 4;      // the lane's piece for even and odd i
    uint32_t vx[PX], vw[PW];
#pragma unroll
    for (int i = 0; i < PX; i++)
      vx[i] = (uint32_t)((wave * PX + i) * 8 + rl) * (uint32_t)a.x_stride + 16u * ((wave * PX + i) & 1 ? po : pe);
#pragma unroll
    for (int i = 0; i < PW; i++)
      vw[i] = (uint32_t)((wave * PW + i) * 8 + rl) * (uint32_t)a.KB + 16u * ((wave * PW + i) & 1 ? po : pe);
    auto load = [&](int st, uint8_t* buf) {
      const int k0 = st * BK;
      const bool e = k0 + 16 * pe >= a.KB, o = k0 + 16 * po >= a.KB;
#pragma unroll
      for (int i = 0; i < PX; i++)
        dma16(rx, buf + (wave * PX + i) * 1024, ((wave * PX + i) & 1 ? o : e) ? kPast : vx[i], (uint32_t)k0);
#pragma unroll
      for (int i = 0; i < PW; i++)
        dma16(rw, buf + BM * BK + (wave * PW + i) * 1024, ((wave * PW + i) & 1 ? o : e) ? kPast : vw[i], (uint32_t)k0);
    };
    // pieces 4 half + 2 j + h of the lane's rows, in their slots (32-row tiles keep r / 2 % 8)
    const int swz = 16 * (h ^ ((r32 >> 1) & 7));
    const int xb = (wm * TI * 32 + r32) * BK, wb = BM * BK + (wn * TJ * 32 + r32) * BK;
    const int ob = XLONG ? xb : wb, ib = XLONG ? wb : xb;
    auto read = [&](const uint8_t* b, int base, int half, int j, int tile) {
      return lds_piece(b, base + (swz ^ (64 * half + 32 * j)) + tile * 32 * BK);
    };
    Acc acc[TJ][TI];
#pragma unroll
    for (int tj = 0; tj < TJ; tj++)
#pragma unroll
      for (int ti = 0; ti < TI; ti++)
#pragma unroll
        for (int i = 0; i < 16; i++) acc[tj][ti][i] = 0;
    // the MFMA of piece j of long-side tile o and short-side tile i (E4M3: two, of the piece's halves;
    // the short side's fp16 is kept for all o)
    uint4 fo[NO][2], fi[NI][2], fn[NI][2];
    auto operand = [](const uint4& u, int e) {
      return TYPE == T_E4M3 ? __builtin_bit_cast(uint4, e4m3_half(u, e)) : u;
    };
    auto mfma = [&](int o, int i, const uint4& u, const uint4& v) {
      const uint4 &x = XLONG ? u : v, &w = XLONG ? v : u;
      Acc& c = XLONG ? acc[i][o] : acc[o][i];
      if constexpr (TYPE == T_INT8)
        c = __builtin_amdgcn_mfma_i32_32x32x32_i8(as_i4(w), as_i4(x), c, 0, 0, 0);
      else if constexpr (TYPE == T_BF16)
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf8(w), as_bf8(x), c, 0, 0, 0);
      else
        c = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(w), as_h8(x), c, 0, 0, 0);
    };
    // Half a stage's MFMAs, with the next half's fragments (half `half` of the stage in nb) read
    // behind them: the short side's into a second set, the long side's each over the one its MFMAs
    // have used, so that both and a large tile's accumulators fit the registers.
    constexpr int NH = TYPE == T_E4M3 ? 2 : 1;               // MFMAs a piece
    auto half_stage = [&](const uint8_t* nb, int half, auto loads) {
#pragma unroll
      for (int i = 0; i < NI; i++)
#pragma unroll
        for (int j = 0; j < 2; j++) fn[i][j] = read(nb, ib, half, j, i);
#pragma unroll
      for (int j = 0; j < 2; j++) {
        uint4 si[NI][NH];
#pragma unroll
        for (int i = 0; i < NI; i++)
#pragma unroll
          for (int e = 0; e < NH; e++) si[i][e] = operand(fi[i][j], e);
#pragma unroll
        for (int o = 0; o < NO; o++) {
#pragma unroll
          for (int e = 0; e < NH; e++) {
            const uint4 so = operand(fo[o][j], e);
#pragma unroll
            for (int i = 0; i < NI; i++) mfma(o, i, so, si[i][e]);
          }
          fo[o][j] = read(nb, ob, half, j, o);
        }
      }
#pragma unroll
      for (int i = 0; i < NI; i++)
#pragma unroll
        for (int j = 0; j < 2; j++) fi[i][j] = fn[i][j];
      interleave<0, 2 * NH * NO * NI, 2 * (NO + NI), decltype(loads)::value>();
      __builtin_amdgcn_sched_barrier(0);
    };
    // stage st in b (its first half already in registers), stage st + 1 in nb; stage st + R goes into b
    auto step = [&](int st, uint8_t* b, const uint8_t* nb) {
      half_stage(b, 1, Int<0>{});
      wait_barrier<(R - 2) * (PX + PW)>();   // stage st + 1 is in, and every wave has read all of stage st
      load(st + R, b);
      half_stage(nb, 0, Int<PX + PW>{});
    };
    Rows rows;
    if (EARLY && !part) load_rows(a, m0, n0, rows);
    load(first, b0);
    load(first + 1, b1);
    if (R > 2) load(first + 2, b2);
    if (!part) load_columns(a, n0, cs);
    wait_barrier<0>();
#pragma unroll
    for (int j = 0; j < 2; j++) {
#pragma unroll
      for (int o = 0; o < NO; o++) fo[o][j] = read(b0, ob, 0, j, o);
#pragma unroll
      for (int i = 0; i < NI; i++) fi[i][j] = read(b0, ib, 0, j, i);
    }
    int st = first;
    if (R == 2) {
      for (; st + 2 <= last; st += 2) {
        step(st, b0, b1);
        step(st + 1, b1, b0);
      }
      if (st < last) step(st, b0, b1);
    } else {
      for (; st + 3 <= last; st += 3) {
        step(st, b0, b1);
        step(st + 1, b1, b2);
        step(st + 2, b2, b0);
      }
      if (st < last) step(st, b0, b1);
      if (st + 1 < last) step(st + 1, b1, b2);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");         // no LDS-DMA in flight from here on
    if (part) {
      store_part(part, acc);
    } else {
      __syncthreads();                       // nobody reads the ring any more
      if (!EARLY) load_rows(a, m0, n0, rows);
      finish(a, m0, n0, b0, b1, cs, rows, acc);
    }
  }

  static __device__ __forceinline__ void load_columns(const Args& a, int n0, float* cs) {
    for (int i = threadIdx.x; i < BN; i += NT) {
      const bool in = n0 + i < a.N;
      cs[i] = in && a.ws ? a.ws[n0 + i] : 1.f;
      cs[BN + i] = in && a.bias ? load16(a.bias, n0 + i, a.bf) : 0.f;
    }
  }

  // A split's sums of a tile: [wave][tile of the wave][quarter][lane], 16 bytes each.
  static constexpr int64_t PART = (int64_t)BM * BN / 16;     // in Acc (16 values)
  static __device__ __forceinline__ uint4* part_at(Acc* part, int tj, int ti) {
    return reinterpret_cast<uint4*>(part) + (((threadIdx.x >> 6) * TJ + tj) * TI + ti) * 256 + (threadIdx.x & 63);
  }
  static __device__ __forceinline__ void store_part(Acc* part, const Acc (&acc)[TJ][TI]) {
#pragma unroll
    for (int tj = 0; tj < TJ; tj++)
#pragma unroll
      for (int ti = 0; ti < TI; ti++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
          uint4 v;
          __builtin_memcpy(&v, reinterpret_cast<const char*>(&acc[tj][ti]) + 16 * q, 16);
          part_at(part, tj, ti)[q * 64] = v;
        }
  }
  // Epilogue: each wave stages its block in 16-bit row pieces, so that global accesses take whole
  // lines.  b0, b1: LDS that nobody else uses.
  static __device__ __forceinline__ void finish(const Args& a, int m0, int n0, uint8_t* b0, uint8_t* b1, const float* cs,
                                                const Rows& rows, const Acc (&acc)[TJ][TI]) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int h = lane >> 5, r32 = lane & 31, wm = wave / WN, wn = wave % WN;
    static_assert(NW / 2 * TI * 32 * RB <= BUF, "the staged blocks must fit two ring buffers");
    uint8_t* ys = (wave < NW / 2 ? b0 : b1) + (wave % (NW / 2)) * TI * 32 * RB;
    const int mw = m0 + wm * TI * 32, nw = wn * TJ * 32;
    auto at = [&](int row, int slot) { return reinterpret_cast<uint4*>(ys + row * RB + 16 * (slot ^ (row & SWAP))); };
    auto sync = [&]() {                                      // the wave's own LDS writes before its reads
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    };
    if (a.res) {
#pragma unroll
      for (int i = 0; i < PASSES; i++)
        *at((i * 64 + lane) / SL, (i * 64 + lane) % SL) =
            make_uint4(rows.res[i][0], rows.res[i][1], rows.res[i][2], rows.res[i][3]);
      sync();
    }
#pragma unroll
    for (int tj = 0; tj < TJ; tj++)
#pragma unroll
      for (int g = 0; g < 2; g++) {
        const int c = nw + tj * 32 + 16 * g + 8 * h, slot = 4 * tj + 2 * g + h;   // the lane's 8 columns after the exchange
        float sw[8], bv[8];
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          *reinterpret_cast<float4*>(sw + e) = *reinterpret_cast<const float4*>(cs + c + e);
          *reinterpret_cast<float4*>(bv + e) = *reinterpret_cast<const float4*>(cs + BN + c + e);
        }
#pragma unroll
        for (int ti = 0; ti < TI; ti++) {
          const int row = ti * 32 + r32;
          float v[8];
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint((float)acc[tj][ti][8 * g + j]),
                                                            __float_as_uint((float)acc[tj][ti][8 * g + 4 + j]), false, false);
            v[j] = __uint_as_float(s[0]);
            v[4 + j] = __uint_as_float(s[1]);
          }
#pragma unroll
          for (int e = 0; e < 8; e++) v[e] = activate(v[e] * rows.sx[ti] * sw[e] + bv[e], a.act);
          if (a.res) {
            float r[8];
            unpack8(*at(row, slot), a.bf, r);
#pragma unroll
            for (int e = 0; e < 8; e++) v[e] += r[e];
          }
          *at(row, slot) = pack8(v, a.bf);
        }
      }
    sync();
#pragma unroll
    for (int i = 0; i < PASSES; i++) {
      const int row = (i * 64 + lane) / SL, ss = (i * 64 + lane) % SL, m = mw + row, n = n0 + nw + ss * 8;
      const uint4 u = *at(row, ss);
      const uint32_t v[4] = {u.x, u.y, u.z, u.w};
      if (m < a.M && n < a.N) store_piece<8>(a.y, m * a.y_stride + n, a.N - n, v);
    }
  }
};

// Tiles of one shape, K in `splits` parts with their sums in `part` (one split: none).
template <int TYPE, int WM, int WN, int TI, int TJ, int R, int OCC>
__global__ void __launch_bounds__(64 * WM * WN, OCC) k_gemm_tile(Args a, int splits, void* part) {
  using T = Tile<TYPE, WM, WN, TI, TJ, R>;
  __shared__ __attribute__((aligned(16))) uint8_t b0[T::BUF];
  __shared__ __attribute__((aligned(16))) uint8_t b1[T::BUF];
  __shared__ __attribute__((aligned(16))) uint8_t b2[R > 2 ? T::BUF : 16];
  __shared__ __attribute__((aligned(16))) float cs[2 * T::BN];
  const int tiles_m = (a.M + T::BM - 1) / T::BM, tiles_n = (a.N + T::BN - 1) / T::BN, tiles = tiles_m * tiles_n;
  const int stages = (a.KB + BK - 1) / BK;
  const int sp = blockIdx.x / tiles, id = blockIdx.x - sp * tiles;
  int tm, tn;
  skel::tile_of(id, tiles, tiles_m, tiles_n, &tm, &tn);
  const int first = (int)((int64_t)stages * sp / splits), last = (int)((int64_t)stages * (sp + 1) / splits);
  typename T::Acc* to = splits > 1 ? static_cast<typename T::Acc*>(part) + ((int64_t)sp * tiles + id) * T::PART : nullptr;
  T::run(a, tm * T::BM, tn * T::BN, b0, b1, b2, cs, first, last, to);
}

// The splits' sums added in order, and the epilogue, four columns a thread: workgroup j of a tile
// takes quarter-tile pieces 4 j ... 4 j + 3 of its waves' 32 x 32 blocks.  Every load goes out
// before the first sum (64 x 3072 in five splits: 4.0 us; with the tile kernel's staged
// epilogue, one workgroup a tile, 7.6).
template <int TYPE, int WM, int WN>
__global__ void __launch_bounds__(256) k_gemm_join(Args a, int splits, const uint4* part) {
  constexpr int BM = WM * 32, BN = WN * 32, GROUPS = WM * WN;
  const int tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + BN - 1) / BN, tiles = tiles_m * tiles_n;
  const int id = blockIdx.x / GROUPS, wave = blockIdx.x - id * GROUPS;
  int tm, tn;
  skel::tile_of(id, tiles, tiles_m, tiles_n, &tm, &tn);
  const int q = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int m = tm * BM + wave / WN * 32 + (lane & 31), n = tn * BN + wave % WN * 32 + 8 * q + 4 * (lane >> 5);
  if (m >= a.M || n >= a.N) return;
  const uint4* from = part + ((int64_t)id * GROUPS + wave) * 256 + threadIdx.x;
  const int64_t next = (int64_t)tiles * GROUPS * 256;
  float sw[4], bv[4];
  uint32_t rr[2] = {0, 0};
  if (a.res) load_piece<4>(a.res, m * a.res_stride + n, a.N - n, rr);
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const bool in = n + j < a.N;
    sw[j] = in && a.ws ? a.ws[n + j] : 1.f;
    bv[j] = in && a.bias ? load16(a.bias, n + j, a.bf) : 0.f;
  }
  const float sx = a.xs ? a.xs[m] : 1.f;
  using Sum = typename Quarter<TYPE>::Sum;
  Sum v = {0, 0, 0, 0};
  for (int s0 = 0; s0 < splits; s0 += 8) {
    uint4 u[8];
#pragma unroll
    for (int s = 0; s < 8; s++)
      u[s] = s0 + s < splits ? from[(s0 + s) * next] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int s = 0; s < 8; s++) v += __builtin_bit_cast(Sum, u[s]);
  }
  float y[4], rv[4];
  unpack4(rr, a.bf, rv);
#pragma unroll
  for (int j = 0; j < 4; j++) y[j] = activate((float)v[j] * sx * sw[j] + bv[j], a.act) + rv[j];
  const uint32_t o[2] = {pack16(y[0], y[1], a.bf), pack16(y[2], y[3], a.bf)};
  store_piece<4>(a.y, m * a.y_stride + n, a.N - n, o);
}

template <int TYPE, int WM, int WN, int TI, int TJ, int R, int OCC>
hipError_t go(const Args& a, int splits, void* part, hipStream_t s) {
  using T = Tile<TYPE, WM, WN, TI, TJ, R>;
  const int64_t tiles = (int64_t)((a.M + T::BM - 1) / T::BM) * ((a.N + T::BN - 1) / T::BN);
  if (!launchable(tiles * splits, T::NT)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_gemm_tile<TYPE, WM, WN, TI, TJ, R, OCC>), dim3((unsigned)(tiles * splits)), dim3(T::NT), 0, s, a,
                     splits, part);
  return hipGetLastError();
}

template <int TYPE, int WM, int WN, int TI, int TJ, int R, int OCC>
hipError_t go_split(const Args& a, int splits, void* part, hipStream_t s) {
  using T = Tile<TYPE, WM, WN, TI, TJ, R>;
  const hipError_t e = go<TYPE, WM, WN, TI, TJ, R, OCC>(a, splits, part, s);
  if (e != hipSuccess || splits == 1) return e;
  static_assert(TI == 1 && TJ == 1, "k_gemm_join takes waves of one 32 x 32 block");
  const int64_t tiles = (int64_t)((a.M + T::BM - 1) / T::BM) * ((a.N + T::BN - 1) / T::BN);
  hipLaunchKernelGGL((k_gemm_join<TYPE, WM, WN>), dim3((unsigned)(tiles * T::NW)), dim3(256), 0, s, a, splits,
                     static_cast<const uint4*>(part));
  return hipGetLastError();
}

// Tiles of 256 x 256, the first `whole` as they are and the rest (a last partial round) in `parts`
// of 128 x 256 or 128 x 128, so that they find all CUs: 4608 x 3072 x 12288 is 3.375 rounds.
template <int TYPE>
__global__ void __launch_bounds__(512, 1) k_gemm_large(Args a, int whole, int parts) {
  using T = Tile<TYPE, 2, 4, 4, 2, 2>;
  using Half = Tile<TYPE, 2, 4, 2, 2, 2>;
  using Fourth = Tile<TYPE, 2, 4, 2, 1, 2>;
  __shared__ __attribute__((aligned(16))) uint8_t b0[T::BUF];
  __shared__ __attribute__((aligned(16))) uint8_t b1[T::BUF];
  __shared__ __attribute__((aligned(16))) float cs[2 * T::BN];
  const int tiles_m = (a.M + T::BM - 1) / T::BM, tiles_n = (a.N + T::BN - 1) / T::BN;
  const int id = blockIdx.x, rest = id - whole;
  const int tile = rest < 0 ? id : whole + rest / parts, part = rest < 0 ? 0 : rest % parts;
  int tm, tn;
  skel::tile_of(tile, tiles_m * tiles_n, tiles_m, tiles_n, &tm, &tn);
  const int m0 = tm * T::BM + (part & 1) * 128, n0 = tn * T::BN + (part >> 1) * 128;
  if (m0 >= a.M || n0 >= a.N) return;
  const int stages = (a.KB + BK - 1) / BK;
  if (rest < 0 || parts == 1) T::run(a, m0, n0, b0, b1, nullptr, cs, 0, stages, nullptr);
  else if (parts == 2) Half::run(a, m0, n0, b0, b1, nullptr, cs, 0, stages, nullptr);
  else Fourth::run(a, m0, n0, b0, b1, nullptr, cs, 0, stages, nullptr);
}

template <int TYPE>
hipError_t go_large(const Args& a, const GemmActPlan& p, hipStream_t s) {
  const int64_t rest = (int64_t)((a.M + 255) / 256) * ((a.N + 255) / 256) - p.whole, blocks = p.whole + rest * p.tail;
  if (!launchable(blocks, 512)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(k_gemm_large<TYPE>, dim3((unsigned)blocks), dim3(512), 0, s, a, p.whole, p.tail);
  return hipGetLastError();
}

template <int TYPE>
hipError_t launch_type(const Args& a, const GemmActPlan& p, void* part, hipStream_t s) {
  switch (p.kind) {
    case GemmActPlan::T64: return go_split<TYPE, 2, 2, 1, 1, 3, 2>(a, p.splits, part, s);
    case GemmActPlan::T64x128: return go_split<TYPE, 2, 4, 1, 1, 3, 2>(a, p.splits, part, s);
    case GemmActPlan::T128x192: return go<TYPE, 4, 2, 1, 3, 3, 1>(a, 1, nullptr, s);
    case GemmActPlan::T128x256: return go<TYPE, 2, 4, 2, 2, 3, 1>(a, 1, nullptr, s);
    case GemmActPlan::LARGE: return go_large<TYPE>(a, p, s);
    default: return hipErrorInvalidValue;
  }
}

int64_t tiles_of(int M, int N, int bm, int bn) { return (int64_t)((M + bm - 1) / bm) * ((N + bn - 1) / bn); }

}  // namespace

// The kernel that costs least, in microseconds fitted to every kernel's time over M = 1 ... 4608,
// N = 1024 ... 12288 and K = 1024 ... 12288 in int8 and bf16, and for E4M3 with constants of its
// own.  Of 114 such sizes in each of the four types the choice is the best kernel or within 9% of it,
// except 65 x 3072 x 3072 in 16 bits (14.8 us, 12.8 in 64 x 128 tiles with more splits).  A stage of
// 128 bytes of K costs a CU its LDS-DMA (0.21 us for each 64 x 64 tile it holds, 0.29 for 64 x 128) but
// no less than the ring's latency with one tile (0.25).  With all CUs at work 128 x 192 tiles take
// 0.7 a stage, 128 x 256 0.95 and 256 x 256 1.72, and less with few.  A split of K costs the sums'
// round trip and a second launch (2.8 us on the GPU, and 3 more that its host work counts).
//
// Both sides, in us without an activation, int8 (M x K x N): few rows / tiles 1 x 3072 x 12288 9.1 / 10.6,
// 17 x 3072 x 12288 9.3 / 10.7, 33 x 3072 x 12288 13.7 / 10.9, 64 x 3072 x 3072 6.8 / 8.1; 64 x 64 / 64 x 128
// tiles 65 x 3072 x 3072 8.1 / 9.6, 512 x 3072 x 3072 13.5 / 11.9; 64 x 128 / 128 x 192 384 x 3072 x 3072
// 11.7 / 17.8, 512 x 3072 x 9216 28.1 / 22.6; 128 x 192 / 128 x 256 the same 22.6 / 25.3,
// 777 x 3072 x 9216 41.3 / 30.6; 128 x 192 / 256 x 256 1536 x 3072 x 3072 22.8 / 29.7,
// 3000 x 12288 x 3072 130 / 128; 128 x 256 / 256 x 256 777 x 3072 x 9216 30.6 / 42.0,
// 4608 x 3072 x 12288 194 / 179; 64 x 12288 x 3072 in 64 x 64 tiles 26.5 whole, 14.8 in five splits.
//
// E4M3: its products take the time of 16-bit ones (twice an 8-bit stage's MFMAs) and the conversion
// to fp16 comes on top, so that the matrix cores and the vector units bound the stages that LDS-DMA
// bounds in the other types.  With the others' constants 777 x 12288 x 3072 took 93 us in 128 x 192
// tiles (64 x 64: 74) and 384 x 6144 x 6144 51 (39).
struct Costs {
  double few, few_rows;                      // few rows: a turn of K, and more for each 16 rows
  double t64, t64_one, t64x128;              // a stage, 64 x 64 tiles with several and one a CU; 64 x 128
  double t192, t192_rest, t192_share;        // a stage with all CUs at work; with few, and more for their share
  double t256, t256_rest, t256_share;
  double large, quarter, quarter_share, half, rest, share;
};
constexpr Costs kCosts{0.19, 0.055, 0.21, 0.25, 0.29, 0.7, 0.4, 0.15, 0.95, 0.5, 0.3, 1.72, 0.65, 0, 0.85, 0.75, 0.95};
constexpr Costs kCostsE4M3{0.2, 0.06, 0.28, 0.32, 0.46, 1.2, 0.75, 0.4, 1.57, 1.0, 0.4, 2.75, 0.65, 0.6, 1.2, 1.2, 1.6};

GemmActPlan plan(int M, int N, int KB, int64_t part_bytes, const Costs& t) {
  const int ncu = resident_workgroups() / 2;
  const double cus = ncu;
  const double S = (KB + BK - 1) / BK;
  GemmActPlan best{};
  double least = 1e30;
  auto consider = [&](int kind, int splits, double cost, int64_t bytes) {
    if (bytes <= part_bytes && cost < least) {
      least = cost;
      best = GemmActPlan{kind, splits, (size_t)bytes, 0, 0};
    }
  };
  if (M <= kFewRows) {
    const int ti = (M + 15) / 16;
    const double c = (N + 15) / 16 / cus, rounds = ceil(c / (ti <= 2 ? 3 : 2));
    consider(GemmActPlan::FEW, 1,
             ceil(S / 4) * ceil(c) * (t.few + t.few_rows * ti) + 3.2 + 0.25 * ti + 0.3 * c + 1.5 * (rounds - 1), 0);
  }
  for (int splits = 1; splits <= 16; splits++) {
    if (splits > 1 && S / splits < 4) break;
    const double st = ceil(S / splits);
    auto join = [&](int64_t bytes) { return splits > 1 ? 5.8 + 0.1 * splits + (double)bytes * 2 / 4e6 : 0.0; };
    const int64_t t64 = tiles_of(M, N, 64, 64), t128 = tiles_of(M, N, 64, 128);
    const double c64 = (double)(t64 * splits) / cus, c128 = ceil((double)(t128 * splits) / cus);
    const int64_t b64 = splits > 1 ? t64 * splits * 64 * 64 * 4 : 0, b128 = splits > 1 ? t128 * splits * 64 * 128 * 4 : 0;
    consider(GemmActPlan::T64, splits, (c64 > 1 ? t.t64 * ceil(c64) * st + 3 : t.t64_one * st + 3.7) + 0.5 * c64 + join(b64),
             b64);
    consider(GemmActPlan::T64x128, splits, t.t64x128 * c128 * st + 4 + c128 + join(b128), b128);
  }
  // rounds of one workgroup a CU, the last with its share of CUs at work
  const double t1 = tiles_of(M, N, 128, 192) / cus, whole1 = floor(t1), rest1 = t1 - whole1;
  consider(GemmActPlan::T128x192, 1,
           whole1 * (t.t192 * S + 8) + (rest1 > 0 ? (t.t192_rest + t.t192_share * rest1) * S + (whole1 > 0 ? 4.5 : 10) : 0), 0);
  const double t2 = tiles_of(M, N, 128, 256) / cus, whole2 = floor(t2), rest2 = t2 - whole2;
  consider(GemmActPlan::T128x256, 1,
           whole2 * (t.t256 * S + 5.5) + (rest2 > 0 ? (t.t256_rest + t.t256_share * rest2) * S + 8 : 0), 0);
  // 256 x 256: a last partial round is cut so that it finds all CUs
  const int64_t tl = tiles_of(M, N, 256, 256), rounds = tl / ncu, rest = tl - rounds * ncu;
  const int tail = rest == 0 ? 0 : 4 * rest <= ncu ? 4 : 2 * rest <= ncu ? 2 : 1;
  const double share = (double)rest / cus;
  const double last = tail == 0   ? 0
                      : tail == 4 ? (t.quarter + t.quarter_share * share) * S + 6.5
                      : tail == 2 ? t.half * S + 11
                                  : (t.rest + t.share * share) * S + 14;
  consider(GemmActPlan::LARGE, 1, rounds * (t.large * S + 6) + last, 0);
  if (best.kind == GemmActPlan::LARGE) {
    best.whole = (int)(tl - rest);
    best.tail = tail;
  }
  return best;
}

}  // namespace gact

GemmActPlan gemm_act_plan(int M, int N, int K, int type, size_t part_bytes) {
  const int eb = type == T_F16 || type == T_BF16 ? 2 : 1;
  return gact::plan(M, N, K * eb, part_bytes > (size_t)1 << 40 ? (int64_t)1 << 40 : (int64_t)part_bytes,
                    type == T_E4M3 ? gact::kCostsE4M3 : gact::kCosts);
}

hipError_t launch_gemm_act(const GemmActArgs& g, hipStream_t s) {
  const int eb = g.type == T_F16 || g.type == T_BF16 ? 2 : 1;
  gact::Args a{};
  a.x = static_cast<const uint8_t*>(g.x);
  a.x_stride = g.x_stride * eb;
  a.xs = g.xs;
  a.w = static_cast<const uint8_t*>(g.w);
  a.ws = g.ws;
  a.bias = g.bias;
  a.res = g.res;
  a.res_stride = g.res_stride;
  a.M = g.M;
  a.N = g.N;
  a.KB = g.K * eb;
  a.act = g.act;
  a.bf = g.out_type == T_BF16;
  a.y = g.y;
  a.y_stride = g.y_stride;
  const GemmActPlan p = gemm_act_plan(g.M, g.N, g.K, g.type, g.part_bytes);
  if (p.kind == GemmActPlan::FEW) return gact::launch_few(a, g.type, s);
  switch (g.type) {
    case T_INT8: return gact::launch_type<T_INT8>(a, p, g.part, s);
    case T_E4M3: return gact::launch_type<T_E4M3>(a, p, g.part, s);
    case T_F16: return gact::launch_type<T_F16>(a, p, g.part, s);
    case T_BF16: return gact::launch_type<T_BF16>(a, p, g.part, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace svdq
