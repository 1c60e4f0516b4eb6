// Block kernels of the matrix product with an epilogue (ep.h has the formulas).
//
// Blocks of BS x BS outputs, 128-byte stages of K, the LDS images, swizzles, fragment reads and MFMA
// schedule of the direct-load GEMM (direct_gemm.h).  What differs:
//
//  * operands have leading dimensions, any M, N and K, and a block may sum only a part of K
//    (`splits`): few output tiles then still fill 256 CUs, and ep_join adds the parts in their order.
//  * three kernels.  gemm_ep_direct: buffer_load … lds as in direct_gemm.h, two stages, 256- and
//    128-wide blocks, for operands whose 16-byte chunks are aligned and never straddle an edge.
//    gemm_ep_ring: the same loads with four stages, 128- and 64-wide, for problems whose CUs hold one
//    block.  gemm_ep_staged: through registers, any alignment and edge, 64-bit addresses, 128- and
//    64-wide.
//  * one shape of stage count: a stage past K reads as zeros (its DMA offsets are out of range, no
//    memory is touched), so one instantiation serves every K.
//  * the matrix instruction's operands are exchanged (it multiplies Bᵀ·Aᵀ), so a lane holds 4
//    consecutive columns of one row: a 32-row band of the wave's tile goes through LDS in fp32
//    with 16-byte writes, and comes back as 8 consecutive columns per lane, where bias,
//    activation and residual are applied and D is stored 16 bytes at a time (whole 128-byte
//    lines per row on 256-wide blocks).  The band is wave-private: no workgroup barrier.
//
// Bounds, measured on MI355X.  256-wide, 8192^3 bf16: 785 us (1400 TFLOP/s), of which the K loop takes
// 725; with bias, gelu_tanh and Z 806 us; 8192 x 8192 x 4096 e4m3 with everything 217 us (2530 TFLOP/s),
// K loop 165.  The rest is the epilogue of four blocks a CU, which no product covers.  64-wide, warm:
// the L2, from which it draws 13 TB/s.  Small: about 4 us of launch, first loads and instruction fetch.
//
// Internal header; one orientation per translation unit.
#pragma once

#include "direct_gemm.h"
#include "ep.h"
#include "staged.h"

namespace tg {
namespace {

// Dᵀ = Bᵀ·Aᵀ on the matrix unit: b supplies the instruction's first operand.
template <int DT, class F>
__device__ __forceinline__ f32x16 mfma32t(F b, F a, f32x16 c) {
  if constexpr (DT == TG_F16 || DT == TG_BF16)
    return mfma32<DT>(b, a, c);
  else
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
        __builtin_bit_cast(i32x8, b), __builtin_bit_cast(i32x8, a), c, DT & 1, (DT & 3) >> 1, 0, 0, 0,
        0);
}

// 128 bits shifted down by `bits` (0 .. , per lane), zeros from above
__device__ __forceinline__ u32x4 shift_down(u32x4 v, uint32_t bits) {
  if (bits & 64) v = u32x4{v[2], v[3], 0, 0};
  if (bits & 32) v = u32x4{v[1], v[2], v[3], 0};
  const uint32_t r = bits & 31;
  v = u32x4{__builtin_amdgcn_alignbit(v[1], v[0], r), __builtin_amdgcn_alignbit(v[2], v[1], r),
            __builtin_amdgcn_alignbit(v[3], v[2], r), v[3] >> r};
  return bits < 128 ? v : u32x4{0, 0, 0, 0};
}

// Fills one operand's LDS stage through registers.  Slot mapping as Operand::load: instruction
// i of wave w fills the 1 KiB block PER·w + i, lane l its bytes 16l .. 16l+15.
template <bool MN, int PER, int DT, int BS>
struct StagedFetch {
  using EL = Elem<DT>;
  static constexpr int E = EL::kBytes, VE = 16 / E;   // elements per chunk
  u32x4 r[PER];

  // instruction i's chunk of a stage
  __device__ __forceinline__ static StagedPlace where(int i, int stage, int wave, int lane) {
    const uint32_t blk = (uint32_t)(PER * wave + i);
    if constexpr (MN) {
      constexpr uint32_t ROWB = BS * E, CH = ROWB / 16, RPB = 1024 / ROWB;
      const uint32_t k = RPB * blk + (uint32_t)lane / CH;
      return staged_place<true>(stage, EL::kBK, VE, (int)k, (int)(((uint32_t)lane % CH) ^ sm_row<SMV, ROWB>(k)));
    } else {
      const uint32_t row = 8u * blk + ((uint32_t)lane >> 3);
      return staged_place<false>(stage, EL::kBK, VE, (int)row, (int)(((uint32_t)lane & 7u) ^ sk<SKV>(row)));
    }
  }
  // base: the block's first element at k = 0 of the block's part of K; rows: rows (K-major) or columns
  // (M/N-major) from there to the operand's end; kl: k of this part.
  // Every load is 16 whole bytes inside the operand (staged.h), so the loads of all stages are alike, no
  // branch hides how many are in flight, and fix() puts the moved chunks right once they are here.
  __device__ __forceinline__ void get(const uint8_t* base, int64_t ld, int rows, int kl, int stage, int wave,
                                      int lane) {
    const int lines = MN ? kl : rows, width = MN ? rows : kl;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      r[i] = load16(base + staged_offset(where(i, stage, wave, lane), ld, lines, width, VE) * E);
  }
  // Moved chunks down to their place, zeros for k past the end.
  __device__ __forceinline__ void fix(int rows, int kl, int stage, int wave, int lane) {
    const int width = MN ? rows : kl;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      r[i] = shift_down(r[i], 8u * E * (uint32_t)staged_back<MN>(where(i, stage, wave, lane), kl, width, VE));
  }
  // Element by element: lines shorter than 16 bytes.
  __device__ __forceinline__ void get_each(const uint8_t* base, int64_t ld, int rows, int kl, int stage, int wave,
                                           int lane) {
    const int lines = MN ? kl : rows, width = MN ? rows : kl;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const StagedPlace at = where(i, stage, wave, lane);
      const uint8_t* p = base + ((int64_t)at.line * ld + at.first) * E;
      const int n = at.line < lines ? width - at.first : 0;
      u32x4 v = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        uint32_t x = 0;
        if (e < n) x = E == 2 ? (uint32_t)((const uint16_t*)p)[e] : (uint32_t)p[e];
        v[e * E / 4] |= x << (8 * E * (e % (4 / E)));
      }
      r[i] = v;
    }
  }
  __device__ __forceinline__ void put(uint8_t* stage, int wave, int lane) const {
#pragma unroll
    for (int i = 0; i < PER; ++i) *(u32x4*)(stage + (wave * PER + i) * 1024 + lane * 16) = r[i];
  }
};

// Waves of a block: 2 x 4, on 64 rows and columns 2 x 2.  (4 waves read a third less of LDS, but one wave
// per SIMD waits for all of it and for its epilogue: 128-wide blocks, 512 x 2048 x 2048, 17.2 -> 19.1 us;
// 256-wide ones, 8192^3 bf16, 781 -> 818.)
constexpr int ep_threads(int bs) { return bs == 64 ? 256 : 512; }

// What a workgroup computes: its block's first row and column, its part of K.
struct EpTile {
  int m0, n0, split, k0, kl;
};
// tile scheduler: contiguous ranges per XCD; parts of K outermost, then grouped tile-rows
template <int BS>
__device__ __forceinline__ EpTile ep_tile(const EpArgs& g) {
  const int nb = (int)gridDim.x;
  int bid = (int)blockIdx.x;
  if ((nb & 7) == 0) bid = (bid & 7) * (nb >> 3) + (bid >> 3);
  const int tiles = g.tiles_m * g.tiles_n;
  EpTile t;
  t.split = bid / tiles;
  bid -= t.split * tiles;
  const int group = kGroupM * g.tiles_n;
  const int first_m = (bid / group) * kGroupM;
  const int gsz = min(g.tiles_m - first_m, kGroupM);
  t.m0 = (first_m + (bid % group) % gsz) * BS;
  t.n0 = ((bid % group) / gsz) * BS;
  t.k0 = t.split * g.k_per_split;
  t.kl = min(g.K - t.k0, g.k_per_split);
  return t;
}

// Epilogue, one 32-row band of the wave's tile at a time.  No wave reads or fills a stage buffer any
// more, so the bands live there: s0 .. s3 are four stage arrays.
// Accumulator element r of tile (i, j): row 32i + lane%32, column 32j + 8(r/4) + 4(lane/32) + r%4.
template <int BS, int WN, int TM, int TN>
__device__ __forceinline__ void ep_store(const EpArgs& g, const EpTile& t, f32x16 (&acc)[TM][TN], int wave,
                                         int lane, int wm, int wn, uint8_t* s0, uint8_t* s1, uint8_t* s2,
                                         uint8_t* s3) {
  constexpr int LDF = WN + 4;   // floats per band row: 16-byte rows, 4 banks apart
  static_assert((BS == 64 ? 1 : 2) * 32 * LDF * 4 <= BS * kRowBytes, "two bands (four waves: one) per stage array");
  float* band = (float*)((wave & 2) ? ((wave & 1) ? s3 : s2) : ((wave & 1) ? s1 : s0)) + (wave >> 2) * 32 * LDF;
  constexpr int LPR = WN / 8, RPP = 64 / LPR;   // lanes per row, rows per pass
  const int bcol = 8 * (lane % LPR), brow = lane / LPR;
  const int col = t.n0 + wn + bcol;
  EpCols cols;
  if (g.splits == 1) ep_cols(g, col, cols);
  // The bands run in a loop, the accumulators moving down a row of tiles each time: unrolled, the
  // epilogue was 250 KB of code, and fetching it took 16 us a 256-wide block.
  auto from_band = [&](int p, float (&v)[8]) {
    const float* src = band + (p * RPP + brow) * LDF + bcol;
    const float4 lo = *(const float4*)src, hi = *(const float4*)(src + 4);
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
  };
  constexpr int NP = 32 / RPP;
  const bool in = col < g.N, half = g.d_t != TG_F32;   // half: 16-bit results
  // residual and row scales: one band ahead of the one being stored
  EpRow ahead[NP];
  auto look = [&](int i) {
    if (g.splits > 1 || !half) return;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int row = t.m0 + wm + 32 * i + brow + p * RPP;
      if (in && row < g.M) ep_row(g, row, col, ahead[p]);
    }
  };
  // (128- and 64-wide blocks share a CU with another and have no registers for it)
  constexpr bool kAhead = BS == 256;
  if (kAhead) look(0);
#pragma unroll 1
  for (int i = 0; i < TM; ++i) {
    const int row0 = t.m0 + wm + 32 * i + brow;
    if (!kAhead) look(i);
    EpRow rows[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) rows[p] = ahead[p];
    if (kAhead && i + 1 < TM) look(i + 1);
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(float4*)(band + (lane & 31) * LDF + 32 * j + 8 * q + 4 * (lane >> 5)) =
            float4{acc[0][j][4 * q], acc[0][j][4 * q + 1], acc[0][j][4 * q + 2], acc[0][j][4 * q + 3]};
#pragma unroll
    for (int k = 0; k + 1 < TM; ++k)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[k][j] = acc[k + 1][j];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    float v[8];
    if (g.splits > 1) {
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        from_band(p, v);
        const int row = row0 + p * RPP;
        if (in && row < g.M)
          ep_put8((uint8_t*)g.part, TG_F32, ((int64_t)t.split * g.M + row) * g.part_ld + col, 8, v);
      }
    } else if (half) {
      ep_with_act(g.act, [&](auto act) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          from_band(p, v);
          const int row = row0 + p * RPP;
          if (in && row < g.M) ep_finish8_16<decltype(act)::value>(g, row, col, cols, rows[p], v);
        }
      });
    } else {
#pragma unroll 1
      for (int p = 0; p < NP; ++p) {
        from_band(p, v);
        const int row = row0 + p * RPP;
        if (in && row < g.M) ep_finish8(g, row, col, cols, v);   // the L2 joins a row's 16-byte pieces
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

// fills one stage's LDS images of both operands from memory
template <bool A_MN, bool B_MN, int DT, int BS, class OA, class OB>
struct DirectLoads {
  using EL = Elem<DT>;
  static constexpr int E = EL::kBytes, BK = EL::kBK;
  OA& oa;
  OB& ob;
  const EpArgs& g;
  int kl, wave;
  uint32_t adv_a, adv_b;
  __device__ __forceinline__ DirectLoads(OA& a, OB& b, const EpArgs& g_, const EpTile& t, int wave_)
      : oa(a), ob(b), g(g_), kl(t.kl), wave(wave_) {
    const uint8_t* pa = g.A + (A_MN ? (int64_t)t.k0 * g.lda + t.m0 : (int64_t)t.m0 * g.lda + t.k0) * E;
    const uint8_t* pb = g.B + (B_MN ? (int64_t)t.k0 * g.ldb + t.n0 : (int64_t)t.n0 * g.ldb + t.k0) * E;
    const int ra = g.M - t.m0, rb = g.N - t.n0;   // rows / columns from here to the end
    // records: from the panel's first element to the last one of this part of K
    oa.bind(pa, (A_MN ? (int64_t)(kl - 1) * g.lda + ra : (int64_t)(min(ra, BS) - 1) * g.lda + kl) * E);
    ob.bind(pb, (B_MN ? (int64_t)(kl - 1) * g.ldb + rb : (int64_t)(min(rb, BS) - 1) * g.ldb + kl) * E);
    adv_a = A_MN ? (uint32_t)(BK * g.lda * E) : (uint32_t)kRowBytes;
    adv_b = B_MN ? (uint32_t)(BK * g.ldb * E) : (uint32_t)kRowBytes;
  }
  // valid bytes of each K row in stage s (K-major operands; 0 for a stage past the end)
  __device__ __forceinline__ void operator()(int s, uint8_t* xa, uint8_t* xb) const {
    const uint32_t lim = (uint32_t)max(0, min(kRowBytes, kl * E - s * kRowBytes));
    oa.template load<true>((uint32_t)s * adv_a, g.lda, xa, wave, lim);
    ob.template load<true>((uint32_t)s * adv_b, g.ldb, xb, wave, lim);
  }
};

// Direct loads, two stages: 256-wide blocks (one workgroup per CU), and 128-wide ones where two
// workgroups share a CU.
template <bool A_MN, bool B_MN, int DT, int BS>
__global__ __launch_bounds__(ep_threads(BS), BS == 128 ? 4 : 2) void gemm_ep_direct(EpArgs g) {
  constexpr int WGM = 2, WGN = ep_threads(BS) / 128;
  // four named stages: their addresses stay compile-time immediates
  __shared__ __attribute__((aligned(1024))) uint8_t sa0[BS * kRowBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sb0[BS * kRowBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sa1[BS * kRowBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sb1[BS * kRowBytes];
  using EL = Elem<DT>;
  using Frag = typename EL::Frag;
  constexpr int NW = WGM * WGN;
  constexpr int WM = BS / WGM, WN = BS / WGN, TM = WM / 32, TN = WN / 32;
  constexpr int PER = BS / 8 / NW;
  constexpr int NS = EL::kSteps;
  static_assert(DT == TG_F16 || DT == TG_BF16 || (DT >= kF8 && DT < kMX), "16-bit or fp8 operands");
  static_assert(!EL::kFp8 || (!A_MN && !B_MN), "fp8 operands are K-contiguous");
  const EpTile t = ep_tile<BS>(g);
  const int tid = (int)threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = (wave / WGN) * WM, wn = (wave % WGN) * WN;
  using OA = Operand<A_MN, TM, PER, DT, BS>;
  using OB = Operand<B_MN, TN, PER, DT, BS>;
  OA oa;
  OB ob;
  oa.init(g.lda, wm, wave, lane);
  ob.init(g.ldb, wn, wave, lane);
  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x16{};
  auto mfmas = [&](const Frag (&a)[TM], const Frag (&b)[TN]) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mfma32t<DT>(b[j], a[i], acc[i][j]);
  };
  Frag a[TM], b[TN];
  constexpr int kReads = OA::kReads + OB::kReads, kMfma = TM * TN;
  using T_ = std::true_type;
  using F_ = std::false_type;
  const DirectLoads<A_MN, B_MN, DT, BS, OA, OB> load_ab(oa, ob, g, t, wave);
  const int KT = (t.kl + EL::kBK - 1) / EL::kBK;   // >= 1
  load_ab(0, sa0, sb0);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  Frag an[TM], bn[TN];
  oa.frags(sa0, 0, a);
  ob.frags(sb0, 0, b);
  load_ab(1, sa1, sb1);
  constexpr int kDma = 2 * PER;

  // fp8: one K step in place, as direct_gemm.h — B's next fragments into spare registers, A
  // tile i's into a[i] once its MFMAs are issued
  auto step_inplace = [&](const uint8_t* xa, const uint8_t* xb, int sn, auto read, auto dma) {
    if constexpr (EL::kFp8) {
      constexpr bool kRead = decltype(read)::value;
      if constexpr (kRead) ob.frags(xb, sn, bn);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = mfma32t<DT>(b[j], a[i], acc[i][j]);
        if constexpr (kRead) oa.frag_tile(xa, sn, i, a[i]);
      }
      constexpr int nra = kRead ? OA::kTileReads : 0, nrb = kRead ? OB::kReads : 0;
      interleave_inplace<TN, kMfma, nra, nrb, decltype(dma)::value ? kDma : 0>();
      if constexpr (kRead) {
#pragma unroll
        for (int j = 0; j < TN; ++j) b[j] = bn[j];
      }
    }
  };
  // one K stage; dma: also load stage kt+2 into the buffer this one frees; next: read the next
  // stage's first fragments
  auto stage = [&](uint8_t* ca, uint8_t* cb, const uint8_t* na, const uint8_t* nb_, int kt, auto dma,
                   auto next) {
    if constexpr (EL::kFp8) {
      step_inplace(ca, cb, 1, T_{}, F_{});
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      if constexpr (decltype(dma)::value) load_ab(kt + 2, ca, cb);
      step_inplace(na, nb_, 0, next, dma);
    } else {
#pragma unroll
      for (int s = 0; s < NS - 1; ++s) {
        oa.frags(ca, s + 1, an);
        ob.frags(cb, s + 1, bn);
        mfmas(a, b);
        interleave<kMfma, kReads, 0>();
#pragma unroll
        for (int i = 0; i < TM; ++i) a[i] = an[i];
#pragma unroll
        for (int j = 0; j < TN; ++j) b[j] = bn[j];
      }
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      if constexpr (decltype(next)::value) {
        oa.frags(na, 0, an);
        ob.frags(nb_, 0, bn);
      }
      if constexpr (decltype(dma)::value) load_ab(kt + 2, ca, cb);
      mfmas(a, b);
      if constexpr (decltype(dma)::value) interleave<kMfma, kReads, kDma>();
      else if constexpr (decltype(next)::value) interleave<kMfma, kReads, 0>();
      if constexpr (decltype(next)::value) {
#pragma unroll
        for (int i = 0; i < TM; ++i) a[i] = an[i];
#pragma unroll
        for (int j = 0; j < TN; ++j) b[j] = bn[j];
      }
    }
  };
  int kt = 0;
  for (; kt + 2 < KT; kt += 2) {   // KT rounded up to even; the last two stages are peeled
    stage(sa0, sb0, sa1, sb1, kt, T_{}, T_{});
    stage(sa1, sb1, sa0, sb0, kt + 1, T_{}, T_{});
  }
  stage(sa0, sb0, sa1, sb1, kt, F_{}, T_{});
  stage(sa1, sb1, sa0, sb0, kt + 1, F_{}, F_{});
  ep_store<BS, WN, TM, TN>(g, t, acc, wave, lane, wm, wn, sa0, sb0, sa1, sb1);
}

// s_waitcnt: at most n vector memory instructions outstanding (n < 64), no LDS read
constexpr int wait_vm(int n) { return (n & 15) | 7 << 4 | (n >> 4) << 14; }

// Direct loads, a ring of four stages (128 KiB on 128-wide blocks): the loads of a stage have three
// stages' time to arrive where two leave one.  For problems of few blocks, whose stages come from far
// away and whose CUs hold one workgroup anyway.
// Stage kt of slot kt % 4, all of whose fragments are in registers: the wave waits until its own loads
// of stage kt + 1 have landed (those of kt + 2 and kt + 3 stay in flight) and meets the others at the
// barrier, so stage kt + 1 is whole and slot kt % 4 free; then the products of stage kt cover the
// reads of all fragments of kt + 1 and the issue of stage kt + 4.  A step at a time, as the two-stage
// kernel reads, every step of a 64-wide block waited for LDS: one wave per SIMD has 32 cycles of
// products a step against about 130 of latency.
// Stages past K read as zeros and touch no memory.
template <bool A_MN, bool B_MN, int DT, int BS>
__global__ __launch_bounds__(ep_threads(BS)) void gemm_ep_ring(EpArgs g) {
  constexpr int WGM = 2, WGN = ep_threads(BS) / 128;
  // one array a stage, A's image and then B's: the compiler tells the loads in flight apart by array
  __shared__ __attribute__((aligned(1024))) uint8_t s0[2 * BS * kRowBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t s1[2 * BS * kRowBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t s2[2 * BS * kRowBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t s3[2 * BS * kRowBytes];
  constexpr int kB = BS * kRowBytes;
  using EL = Elem<DT>;
  using Frag = typename EL::Frag;
  constexpr int NW = WGM * WGN;
  constexpr int WM = BS / WGM, WN = BS / WGN, TM = WM / 32, TN = WN / 32;
  constexpr int PER = BS / 8 / NW;
  constexpr int NS = EL::kSteps;
  static_assert(DT == TG_F16 || DT == TG_BF16 || (DT >= kF8 && DT < kMX), "16-bit or fp8 operands");
  static_assert(!EL::kFp8 || (!A_MN && !B_MN), "fp8 operands are K-contiguous");
  const EpTile t = ep_tile<BS>(g);
  const int tid = (int)threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = (wave / WGN) * WM, wn = (wave % WGN) * WN;
  using OA = Operand<A_MN, TM, PER, DT, BS>;
  using OB = Operand<B_MN, TN, PER, DT, BS>;
  OA oa;
  OB ob;
  oa.init(g.lda, wm, wave, lane);
  ob.init(g.ldb, wn, wave, lane);
  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x16{};
  auto mfmas = [&](const Frag (&a)[TM], const Frag (&b)[TN]) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mfma32t<DT>(b[j], a[i], acc[i][j]);
  };
  constexpr int kReads = OA::kReads + OB::kReads, kMfma = TM * TN, kDma = 2 * PER;
  const DirectLoads<A_MN, B_MN, DT, BS, OA, OB> load_ab(oa, ob, g, t, wave);
  const int KT = (t.kl + EL::kBK - 1) / EL::kBK;   // >= 1
  // the barrier alone: __syncthreads would wait for every load
  auto meet = [&](auto n) {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_vm(decltype(n)::value));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  load_ab(0, s0, s0 + kB);
  load_ab(1, s1, s1 + kB);
  load_ab(2, s2, s2 + kB);
  load_ab(3, s3, s3 + kB);
  meet(std::integral_constant<int, 3 * kDma>{});
  Frag fa[2][NS][TM], fb[2][NS][TN];   // fragments of two stages, the even and the odd one
  auto read = [&](const uint8_t* st, Frag (&x)[NS][TM], Frag (&y)[NS][TN]) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      oa.frags(st, s, x[s]);
      ob.frags(st + kB, s, y[s]);
    }
  };
  read(s0, fa[0], fb[0]);
  auto stage = [&](uint8_t* cur, const uint8_t* next, int kt, auto odd) {
    constexpr int p = decltype(odd)::value;
    meet(std::integral_constant<int, 2 * kDma>{});
    read(next, fa[1 - p], fb[1 - p]);
    load_ab(kt + 4, cur, cur + kB);
#pragma unroll
    for (int s = 0; s < NS; ++s) mfmas(fa[p][s], fb[p][s]);
    interleave<kMfma * NS, kReads * NS, kDma>();
  };
  constexpr std::integral_constant<int, 0> even{};
  constexpr std::integral_constant<int, 1> odd{};
  // No way out of the middle of a round: the compiler would count the loads of every exit as possibly
  // in flight at the loop's head, and wait for all of them there.
  int kt = 0;
  for (; kt + 4 <= KT; kt += 4) {
    stage(s0, s1, kt, even);
    stage(s1, s2, kt + 1, odd);
    stage(s2, s3, kt + 2, even);
    stage(s3, s0, kt + 3, odd);
  }
  if (kt < KT) {
    stage(s0, s1, kt, even);
    if (kt + 1 < KT) {
      stage(s1, s2, kt + 1, odd);
      if (kt + 2 < KT) stage(s2, s3, kt + 2, even);
    }
  }
  // the zero stages still on their way must land before the epilogue takes the buffers
  meet(std::integral_constant<int, 0>{});
  ep_store<BS, WN, TM, TN>(g, t, acc, wave, lane, wm, wn, s0, s1, s2, s3);
}

// Operands through registers, two stages ahead of the one computed: one register set each for the even
// and the odd stage.
template <bool A_MN, bool B_MN, int DT, int BS>
__global__ __launch_bounds__(ep_threads(BS), BS == 128 ? 4 : 2) void gemm_ep_staged(EpArgs g) {
  constexpr int WGM = 2, WGN = ep_threads(BS) / 128;
  __shared__ __attribute__((aligned(1024))) uint8_t sa0[BS * kRowBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sb0[BS * kRowBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sa1[BS * kRowBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sb1[BS * kRowBytes];
  using EL = Elem<DT>;
  using Frag = typename EL::Frag;
  constexpr int NW = WGM * WGN;
  constexpr int WM = BS / WGM, WN = BS / WGN, TM = WM / 32, TN = WN / 32;
  constexpr int PER = BS / 8 / NW;
  constexpr int NS = EL::kSteps;
  static_assert(DT == TG_F16 || DT == TG_BF16 || (DT >= kF8 && DT < kMX), "16-bit or fp8 operands");
  static_assert(!EL::kFp8 || (!A_MN && !B_MN), "fp8 operands are K-contiguous");
  const EpTile t = ep_tile<BS>(g);
  const int tid = (int)threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = (wave / WGN) * WM, wn = (wave % WGN) * WN;
  using OA = Operand<A_MN, TM, PER, DT, BS>;
  using OB = Operand<B_MN, TN, PER, DT, BS>;
  OA oa;
  OB ob;
  oa.init(g.lda, wm, wave, lane);
  ob.init(g.ldb, wn, wave, lane);
  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x16{};
  auto mfmas = [&](const Frag (&a)[TM], const Frag (&b)[TN]) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mfma32t<DT>(b[j], a[i], acc[i][j]);
  };
  Frag a[TM], b[TN];
  constexpr int E = EL::kBytes;
  const uint8_t* pa = g.A + (A_MN ? (int64_t)t.k0 * g.lda + t.m0 : (int64_t)t.m0 * g.lda + t.k0) * E;
  const uint8_t* pb = g.B + (B_MN ? (int64_t)t.k0 * g.ldb + t.n0 : (int64_t)t.n0 * g.ldb + t.k0) * E;
  const int ra = g.M - t.m0, rb = g.N - t.n0;   // rows / columns from here to the end
  const int KT = (t.kl + EL::kBK - 1) / EL::kBK;   // >= 1
  StagedFetch<A_MN, PER, DT, BS> fa[2];
  StagedFetch<B_MN, PER, DT, BS> fb[2];
  auto compute = [&](const uint8_t* xa, const uint8_t* xb) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      oa.frags(xa, s, a);
      ob.frags(xb, s, b);
      mfmas(a, b);
    }
  };
  constexpr int VE = 16 / E;
  if (g.K < VE || (A_MN && g.M < VE) || (B_MN && g.N < VE)) {
    // one stage after the other
    for (int kt = 0; kt < KT; ++kt) {
      fa[0].get_each(pa, g.lda, ra, t.kl, kt, wave, lane);
      fb[0].get_each(pb, g.ldb, rb, t.kl, kt, wave, lane);
      __syncthreads();
      fa[0].put(sa0, wave, lane);
      fb[0].put(sb0, wave, lane);
      __syncthreads();
      compute(sa0, sb0);
    }
    __syncthreads();
  } else {
    // stages past the last load what is not used
    auto get = [&](auto q, int s) {
      constexpr int set = decltype(q)::value;
      fa[set].get(pa, g.lda, ra, t.kl, s, wave, lane);
      fb[set].get(pb, g.ldb, rb, t.kl, s, wave, lane);
      __builtin_amdgcn_sched_barrier(0);   // on their way before the stage's products
    };
    const bool edge_a = A_MN && ra < BS, edge_b = B_MN && rb < BS;
    auto put = [&](auto q, int s, uint8_t* xa, uint8_t* xb) {
      constexpr int set = decltype(q)::value;
      if (edge_a || s + 1 >= KT) fa[set].fix(ra, t.kl, s, wave, lane);
      if (edge_b || s + 1 >= KT) fb[set].fix(rb, t.kl, s, wave, lane);
      fa[set].put(xa, wave, lane);
      fb[set].put(xb, wave, lane);
    };
    constexpr std::integral_constant<int, 0> S0{};
    constexpr std::integral_constant<int, 1> S1{};
    get(S0, 0);
    get(S1, 1);
    put(S0, 0, sa0, sb0);
    __syncthreads();
    // stage kt from (ca, cb); its registers, set `q`, take stage kt + 2, and stage kt + 1, loaded a stage
    // ago, goes to (na, nb) after it
    auto stage = [&](const uint8_t* ca, const uint8_t* cb, uint8_t* na, uint8_t* nb, int kt, auto q, auto next) {
      get(q, kt + 2);
      compute(ca, cb);
      put(next, kt + 1, na, nb);
      __syncthreads();
    };
    int kt = 0;
    for (; kt + 2 <= KT; kt += 2) {
      stage(sa0, sb0, sa1, sb1, kt, S0, S1);
      stage(sa1, sb1, sa0, sb0, kt + 1, S1, S0);
    }
    if (kt < KT) stage(sa0, sb0, sa1, sb1, kt, S0, S1);
  }
  ep_store<BS, WN, TM, TN>(g, t, acc, wave, lane, wm, wn, sa0, sb0, sa1, sb1);
}

template <bool A_MN, bool B_MN, int DT>
hipError_t launch_ep_one(const EpArgs& g, const EpKernel& k, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)g.tiles_m * g.tiles_n * g.splits)), block(ep_threads(k.bs));
  if (k.staged) {
    if (k.bs == 64) hipLaunchKernelGGL((gemm_ep_staged<A_MN, B_MN, DT, 64>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((gemm_ep_staged<A_MN, B_MN, DT, 128>), grid, block, 0, s, g);
  } else if (k.ring) {
    if (k.bs == 64) hipLaunchKernelGGL((gemm_ep_ring<A_MN, B_MN, DT, 64>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((gemm_ep_ring<A_MN, B_MN, DT, 128>), grid, block, 0, s, g);
  } else {
    if (k.bs == 256) hipLaunchKernelGGL((gemm_ep_direct<A_MN, B_MN, DT, 256>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((gemm_ep_direct<A_MN, B_MN, DT, 128>), grid, block, 0, s, g);
  }
  return hipGetLastError();
}

template <bool A_MN, bool B_MN>
hipError_t launch_ep_layout(const EpArgs& g, int dtype, const EpKernel& k, hipStream_t s) {
  return dtype == TG_F16 ? launch_ep_one<A_MN, B_MN, TG_F16>(g, k, s)
                         : launch_ep_one<A_MN, B_MN, TG_BF16>(g, k, s);
}

}  // namespace
}  // namespace tg
