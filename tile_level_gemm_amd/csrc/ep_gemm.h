// Block kernels of the matrix product with an epilogue (ep.h has the formulas).
//
// Blocks of BS x BS outputs by 8 waves (2 x 4), 128-byte stages of K, the LDS images, swizzles,
// fragment reads and MFMA schedule of the direct-load GEMM (direct_gemm.h).  What differs:
//
//  * operands have leading dimensions, any M, N and K, and a block may sum only a part of K
//    (`splits`): few output tiles then still fill 256 CUs, and ep_join adds the parts in
//    their order.
//  * two ways to fill a stage.  Direct: buffer_load … lds as in direct_gemm.h, for operands
//    whose 16-byte chunks are aligned and never straddle an edge.  Staged: each lane loads the
//    16-byte chunk of the same physical slot into registers (any alignment, element by
//    element at an edge, 64-bit addresses) and writes it to LDS after the current stage's
//    MFMAs; it serves every other operand.
//  * one stage-count shape: the count is rounded up to even and a stage past K reads as
//    zeros (its DMA offsets are out of range, no memory is touched), so one instantiation
//    serves every K at the cost of at most one stage of MFMAs.
//  * the matrix instruction's operands are exchanged (it multiplies Bᵀ·Aᵀ), so a lane holds 4
//    consecutive columns of one row: a 32-row band of the wave's tile goes through LDS in fp32
//    with 16-byte writes, and comes back as 8 consecutive columns per lane, where bias,
//    activation and residual are applied and D is stored 16 bytes at a time (whole 128-byte
//    lines per row on 256-wide blocks).  The band is wave-private: no workgroup barrier.
//
// Internal header; one orientation per translation unit.
#pragma once

#include "direct_gemm.h"
#include "ep.h"

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

// Fills one operand's LDS stage through registers.  Slot mapping as Operand::load: instruction
// i of wave w fills the 1 KiB block PER·w + i, lane l its bytes 16l .. 16l+15.
template <bool MN, int PER, int DT, int BS>
struct StagedFetch {
  using EL = Elem<DT>;
  static constexpr int E = EL::kBytes, VE = 16 / E;   // elements per chunk
  u32x4 r[PER];

  // base: the block's first element at k = 0 of the block's part of K; rows: valid rows (K-major)
  // or columns (M/N-major) of the block; kl: valid k.
  __device__ __forceinline__ void get(const uint8_t* base, int64_t ld, int rows, int kl, int stage,
                                      int wave, int lane) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t blk = (uint32_t)(PER * wave + i);
      int64_t off;   // elements
      int n;         // valid elements of the chunk
      if constexpr (MN) {
        constexpr uint32_t ROWB = BS * E, CH = ROWB / 16, RPB = 1024 / ROWB;
        const uint32_t k = RPB * blk + (uint32_t)lane / CH;
        const uint32_t c = ((uint32_t)lane % CH) ^ sm<SMV>(k);
        const int kk = stage * EL::kBK + (int)k;
        off = (int64_t)kk * ld + c * VE;
        n = kk < kl ? rows - (int)(c * VE) : 0;
      } else {
        const uint32_t row = 8u * blk + ((uint32_t)lane >> 3);
        const uint32_t c = ((uint32_t)lane & 7u) ^ sk<SKV>(row);
        const int k = stage * EL::kBK + (int)(c * VE);
        off = (int64_t)row * ld + k;
        n = (int)row < rows ? kl - k : 0;
      }
      const uint8_t* p = base + off * E;
      u32x4 v = {0, 0, 0, 0};
      if (n >= VE) {
        v = load16(p);
      } else if (n > 0) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          uint32_t x = 0;
          if (e < n) x = E == 2 ? (uint32_t)((const uint16_t*)p)[e] : (uint32_t)p[e];
          v[e * E / 4] |= x << (8 * E * (e % (4 / E)));
        }
      }
      r[i] = v;
    }
  }
  __device__ __forceinline__ void put(uint8_t* stage, int wave, int lane) const {
#pragma unroll
    for (int i = 0; i < PER; ++i) *(u32x4*)(stage + (wave * PER + i) * 1024 + lane * 16) = r[i];
  }
};

template <bool A_MN, bool B_MN, int DT, int BS, bool STAGED>
__device__ __forceinline__ void ep_body(const EpArgs& g) {
  using EL = Elem<DT>;
  using Frag = typename EL::Frag;
  constexpr int WGM = 2, WGN = 4, NW = WGM * WGN;
  constexpr int WM = BS / WGM, WN = BS / WGN, TM = WM / 32, TN = WN / 32;
  constexpr int PER = BS / 8 / NW;
  constexpr int E = EL::kBytes, BK = EL::kBK, NS = EL::kSteps;
  static_assert(DT == TG_F16 || DT == TG_BF16 || (DT >= kF8 && DT < kMX), "16-bit or fp8 operands");
  static_assert(!EL::kFp8 || (!A_MN && !B_MN), "fp8 operands are K-contiguous");
  // four named stages: their addresses stay compile-time immediates
  __shared__ __attribute__((aligned(1024))) uint8_t sa0[BS * kRowBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sb0[BS * kRowBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sa1[BS * kRowBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sb1[BS * kRowBytes];

  // tile scheduler: contiguous ranges per XCD; parts of K outermost, then grouped tile-rows
  const int nb = (int)gridDim.x;
  int bid = (int)blockIdx.x;
  if ((nb & 7) == 0) bid = (bid & 7) * (nb >> 3) + (bid >> 3);
  const int tiles = g.tiles_m * g.tiles_n;
  const int split = bid / tiles;
  bid -= split * tiles;
  const int group = kGroupM * g.tiles_n;
  const int first_m = (bid / group) * kGroupM;
  const int gsz = min(g.tiles_m - first_m, kGroupM);
  const int tm = first_m + (bid % group) % gsz;
  const int tn = (bid % group) / gsz;
  const int m0 = tm * BS, n0 = tn * BS;
  const int k0 = split * g.k_per_split;
  const int kl = min(g.K - k0, g.k_per_split);

  const int tid = (int)threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = (wave / WGN) * WM, wn = (wave % WGN) * WN;

  using OA = Operand<A_MN, TM, PER, DT, BS>;
  using OB = Operand<B_MN, TN, PER, DT, BS>;
  OA oa;
  OB ob;
  oa.init(g.lda, wm, wave, lane);
  ob.init(g.ldb, wn, wave, lane);
  const uint8_t* pa = g.A + (A_MN ? (int64_t)k0 * g.lda + m0 : (int64_t)m0 * g.lda + k0) * E;
  const uint8_t* pb = g.B + (B_MN ? (int64_t)k0 * g.ldb + n0 : (int64_t)n0 * g.ldb + k0) * E;
  const int ra = g.M - m0, rb = g.N - n0;   // rows / columns from here to the end

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
  const int KT = (kl + BK - 1) / BK;   // >= 1
  constexpr int kMfma = TM * TN;
  constexpr int kReads = OA::kReads + OB::kReads;
  using T_ = std::true_type;
  using F_ = std::false_type;
  Frag a[TM], b[TN];

  if constexpr (STAGED) {
    StagedFetch<A_MN, PER, DT, BS> fa;
    StagedFetch<B_MN, PER, DT, BS> fb;
    auto get = [&](int s) {
      fa.get(pa, g.lda, ra, kl, s, wave, lane);
      fb.get(pb, g.ldb, rb, kl, s, wave, lane);
    };
    auto compute = [&](const uint8_t* xa, const uint8_t* xb) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        oa.frags(xa, s, a);
        ob.frags(xb, s, b);
        mfmas(a, b);
      }
    };
    get(0);
    fa.put(sa0, wave, lane);
    fb.put(sb0, wave, lane);
    __syncthreads();
    // stage kt from (ca, cb); stage kt+1 travels to registers meanwhile and to (na, nb_) after
    auto stage = [&](const uint8_t* ca, const uint8_t* cb, uint8_t* na, uint8_t* nb_, int kt) {
      const bool more = kt + 1 < KT;
      if (more) get(kt + 1);
      compute(ca, cb);
      if (more) {
        fa.put(na, wave, lane);
        fb.put(nb_, wave, lane);
      }
      __syncthreads();
    };
    for (int kt = 0; kt < KT; kt += 2) {
      stage(sa0, sb0, sa1, sb1, kt);
      if (kt + 1 < KT) stage(sa1, sb1, sa0, sb0, kt + 1);
    }
  } else {
    // records: from the panel's first element to the last one of this part of K
    oa.bind(pa, (A_MN ? (int64_t)(kl - 1) * g.lda + ra : (int64_t)(min(ra, BS) - 1) * g.lda + kl) * E);
    ob.bind(pb, (B_MN ? (int64_t)(kl - 1) * g.ldb + rb : (int64_t)(min(rb, BS) - 1) * g.ldb + kl) * E);
    const uint32_t adv_a = A_MN ? (uint32_t)(BK * g.lda * E) : (uint32_t)kRowBytes;
    const uint32_t adv_b = B_MN ? (uint32_t)(BK * g.ldb * E) : (uint32_t)kRowBytes;
    // valid bytes of each K row in stage s (K-major operands; 0 for a stage past the end)
    auto lim = [&](int s) -> uint32_t { return (uint32_t)max(0, min(kRowBytes, kl * E - s * kRowBytes)); };
    auto load_ab = [&](int s, uint8_t* xa, uint8_t* xb) {
      oa.template load<true>((uint32_t)s * adv_a, g.lda, xa, wave, lim(s));
      ob.template load<true>((uint32_t)s * adv_b, g.ldb, xb, wave, lim(s));
    };
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
  }

  // Epilogue, one 32-row band of the wave's tile at a time.  No wave reads a stage buffer after
  // the last barrier, so the bands live there: two wave regions in each of the four arrays.
  // Accumulator element r of tile (i, j): row 32i + lane%32, column 32j + 8(r/4) + 4(lane/32) + r%4.
  constexpr int LDF = WN + 4;   // floats per band row: 16-byte rows, 4 banks apart
  static_assert(2 * 32 * LDF * 4 <= BS * kRowBytes, "two bands per stage array");
  float* band = (float*)((wave & 2) ? ((wave & 1) ? sb1 : sa1) : ((wave & 1) ? sb0 : sa0)) +
                (wave >> 2) * 32 * LDF;
  constexpr int LPR = WN / 8, RPP = 64 / LPR;   // lanes per row, rows per pass
  const int bcol = 8 * (lane % LPR), brow = lane / LPR;
  const int col = n0 + wn + bcol;
  EpCols cols;
  if (g.splits == 1) ep_cols(g, col, cols);
  // The bands run in a loop whose only unrolled part is the write from the accumulators: unrolled
  // whole, the epilogue was 250 KB of code, and fetching it took 16 us a 256-wide block.
  auto to_band = [&](auto I) {
    constexpr int i = decltype(I)::value < TM ? decltype(I)::value : 0;   // compile-time: registers
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(float4*)(band + (lane & 31) * LDF + 32 * j + 8 * q + 4 * (lane >> 5)) =
            float4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
  };
  auto from_band = [&](int p, float (&v)[8]) {
    const float* src = band + (p * RPP + brow) * LDF + bcol;
    const float4 lo = *(const float4*)src, hi = *(const float4*)(src + 4);
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
  };
  constexpr int NP = 32 / RPP;
  const bool even = ep_even(g), in = col < g.N;
  // residual and row scales: one band ahead of the one being stored
  EpRow ahead[NP];
  auto look = [&](int i) {
    if (g.splits > 1 || !even) return;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int row = m0 + wm + 32 * i + brow + p * RPP;
      if (in && row < g.M) ep_row(g, row, col, ahead[p]);
    }
  };
  look(0);
#pragma unroll 1
  for (int i = 0; i < TM; ++i) {
    const int row0 = m0 + wm + 32 * i + brow;
    EpRow rows[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) rows[p] = ahead[p];
    if (i + 1 < TM) look(i + 1);
    if (i == 0) to_band(std::integral_constant<int, 0>{});
    else if (i == 1) to_band(std::integral_constant<int, 1>{});
    else if (i == 2) to_band(std::integral_constant<int, 2>{});
    else to_band(std::integral_constant<int, 3>{});
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
          ep_put8((uint8_t*)g.part, TG_F32, ((int64_t)split * g.M + row) * g.part_ld + col, 8, v);
      }
    } else if (even) {
      ep_with_act(g.act, [&](auto act) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          from_band(p, v);
          const int row = row0 + p * RPP;
          if (in && row < g.M) ep_finish8_even<decltype(act)::value>(g, row, col, cols, rows[p], v);
        }
      });
    } else {
#pragma unroll 1
      for (int p = 0; p < NP; ++p) {
        from_band(p, v);
        const int row = row0 + p * RPP;
        if (in && row < g.M) ep_finish8(g, row, col, cols, v);   // fp32 or ragged: the L2 joins the pieces
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

template <bool A_MN, bool B_MN, int DT, int BS>
__global__ __launch_bounds__(512) void gemm_ep_direct(EpArgs g) {
  ep_body<A_MN, B_MN, DT, BS, false>(g);
}
template <bool A_MN, bool B_MN, int DT>
__global__ __launch_bounds__(512) void gemm_ep_staged(EpArgs g) {
  ep_body<A_MN, B_MN, DT, 128, true>(g);
}

template <bool A_MN, bool B_MN, int DT>
hipError_t launch_ep_one(const EpArgs& g, int bs, bool staged, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)g.tiles_m * g.tiles_n * g.splits)), block(512);
  if (staged) hipLaunchKernelGGL((gemm_ep_staged<A_MN, B_MN, DT>), grid, block, 0, s, g);
  else if (bs == 256) hipLaunchKernelGGL((gemm_ep_direct<A_MN, B_MN, DT, 256>), grid, block, 0, s, g);
  else hipLaunchKernelGGL((gemm_ep_direct<A_MN, B_MN, DT, 128>), grid, block, 0, s, g);
  return hipGetLastError();
}

template <bool A_MN, bool B_MN>
hipError_t launch_ep_layout(const EpArgs& g, int dtype, int bs, bool staged, hipStream_t s) {
  return dtype == TG_F16 ? launch_ep_one<A_MN, B_MN, TG_F16>(g, bs, staged, s)
                         : launch_ep_one<A_MN, B_MN, TG_BF16>(g, bs, staged, s);
}

}  // namespace
}  // namespace tg
