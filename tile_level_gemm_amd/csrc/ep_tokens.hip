// Product with an epilogue for few rows (ep.h has the formulas): a stream of weights.
//
// Bound by reading B once; A is small and comes from the caches.  A workgroup's waves take K steps
// in turn, 16 waves with 8 KB of B each in flight in registers before their first product, then the
// waves' sums meet in LDS, are added in their order and finished with the epilogue operands that were
// loaded first of all.  A CU draws about 26 GB/s from HBM this way whatever its waves ask for (131 KB:
// 5 us), so the columns are cut until every CU has some.
//
//   B [N][K] (K-major): a step is 128 bytes of K of 16 columns (32 for N >= 8192: A is read half as
//     often).  Lane (n = l%16, g = l/16) loads bytes 32g .. 32g+31 of its column, so four lanes read one
//     whole line; the matrix instruction (16x16x32 for 16-bit, 16x16x128 for fp8) takes K in that order,
//     for A and B alike (a sum does not care).  For small N the workgroup owns 8 or 4 columns and the
//     other lanes load nothing: more CUs, no parts to join.
//   B [K][N]: a step is 32 k-rows of 32 columns.  Where that leaves CUs without work and a workgroup
//     with much, K is cut into parts that ep_join adds.  Lane (j, g) loads columns 2j, 2j+1 of k-rows
//     8g .. 8g+7 (16 lanes read 64 bytes of a row) and turns the 8 pairs into two K-vectors with
//     byte permutes; column 2j + c is column j of instruction c.  64-byte runs rather than 128: twice
//     the workgroups for the same N, and the other half of a line is read on the same XCD.
//
// The instruction's operands are exchanged (Bᵀ·Aᵀ), so a lane holds 4 consecutive columns of one row.
// Any alignment, leading dimension and K: the last partial step loads element by element.
//
// Measured, weights from HBM: 1 x 4096 x 4096 bf16 8.5 us (8 waves with twice as much each 9.3), 1 x 8192 x
// 8192 25.8 us (5.2 TB/s), 16 x 8192 x 4096 e4m3 9.8 us; about 4 us of each are launch and first bytes.
#include "direct_gemm.h"
#include "ep.h"

namespace tg {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;

template <int DT, class F>
__device__ __forceinline__ f32x4 mfma16t(F b, F a, f32x4 c) {
  if constexpr (DT == TG_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), c, 0, 0, 0);
  else if constexpr (DT == TG_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i32x8, b), __builtin_bit_cast(i32x8, a),
                                                            c, DT & 1, (DT & 3) >> 1, 0, 0, 0, 0);
}

// 16 bytes of a K-contiguous row, n valid elements of E bytes from p on (n <= 0: none, nothing is read)
template <int E>
__device__ __forceinline__ u32x4 k_chunk(const uint8_t* p, int n) {
  constexpr int VE = 16 / E;
  if (n >= VE) return load16(p);
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    uint32_t x = 0;
    if (e < n) x = E == 2 ? (uint32_t)((const uint16_t*)p)[e] : (uint32_t)p[e];
    v[e * E / 4] |= x << (8 * E * (e % (4 / E)));
  }
  return v;
}
// the same of an operand whose rows run along the other axis: element e at p[e·ld]
__device__ __forceinline__ u32x4 k_gather(const uint16_t* p, int64_t ld, int n) {
  u32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t lo = 2 * e < n ? p[2 * e * ld] : 0, hi = 2 * e + 1 < n ? p[(2 * e + 1) * ld] : 0;
    v[e] = lo | hi << 16;
  }
  return v;
}
struct __attribute__((packed, aligned(2))) Bytes4 { uint32_t v; };

// MT: row tiles of 16.  blockDim.x / 64 waves.
// NI: column tiles of 16.
template <bool A_MN, bool B_MN, int DT, int MT, int NI>
__global__ __launch_bounds__(1024) void gemm_ep_tokens(EpArgs g) {
  using EL = Elem<DT>;
  constexpr int E = EL::kBytes;
  static_assert(!B_MN || NI == 2, "a lane's two columns");
  constexpr int CN = 16 * NI;                   // most columns of a workgroup
  constexpr int KS = B_MN ? 32 : 128 / E;       // K of a step
  constexpr int KI = E == 2 ? 32 : 128;         // K of an instruction
  constexpr int NF = KS / KI;                   // instructions of a step along K
  constexpr int U = MT == 1 && (B_MN || NI == 1) ? 4 : 2;   // steps in flight
  using Frag = typename EL::Frag;               // one instruction's operand: 8 16-bit values, 32 fp8
  constexpr int LD = CN + 1;
  __shared__ float red[16][MT * 16][LD];

  const int nb = (int)gridDim.x;
  int bid = (int)blockIdx.x;
  if ((nb & 7) == 0) bid = (bid & 7) * (nb >> 3) + (bid >> 3);
  const int blocks_n = (g.N + g.cn - 1) / g.cn;
  const int split = bid / blocks_n;
  const int n0 = (bid - split * blocks_n) * g.cn;
  const int n1 = min(g.N, n0 + g.cn);
  const int W = (int)blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = (int)threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  const int kb = split * g.k_per_split;         // this part of K
  const int K = min(g.K - kb, g.k_per_split), T = (K + KS - 1) / KS, full = K / KS;

  // this thread's first output, and what its epilogue reads: on the way while the sum is taken
  const int orow = (int)threadIdx.x / CN, ocol = n0 + (int)threadIdx.x % CN;
  EpOne pre{};
  if (g.splits == 1 && orow < g.M && orow < 16 * MT && ocol < n1) ep_one(g, orow, ocol, pre);

  // what a lane loads of B in a step, before it is made into fragments
  struct Raw {
    uint32_t r[B_MN ? 8 : NI * 8];
  };
  const int col = n0 + (B_MN ? 2 * li : li);
  const int nc = n1 - col;   // valid columns from this lane's first on
  // k of the lane's first element in a step (B_MN: k-rows; K-major: a run of 32 bytes)
  const int kl = B_MN ? 8 * lg : lg * (32 / E);
  const uint8_t* pb = g.B + (B_MN ? (int64_t)(kb + kl) * g.ldb + col : (int64_t)col * g.ldb + kb + kl) * E;
  const uint8_t* pa = g.A + (A_MN ? (int64_t)kb * g.lda : (int64_t)kb) * E;
  auto load_b = [&](int step, auto partial, Raw& x) {
    constexpr bool kPartial = decltype(partial)::value;
    const int k0 = step * KS, left = K - k0 - kl;
    if constexpr (B_MN) {
      const uint8_t* p = pb + (int64_t)k0 * g.ldb * 2;
#pragma unroll
      for (int e = 0; e < 8; ++e, p += g.ldb * 2) {
        uint32_t v = 0;
        if (nc >= 2 && (!kPartial || e < left)) v = ((const Bytes4*)p)->v;
        else if (nc == 1 && (!kPartial || e < left)) v = *(const uint16_t*)p;
        x.r[e] = v;
      }
    } else {
#pragma unroll
      for (int c = 0; c < NI; ++c) {
        const uint8_t* p = pb + ((int64_t)16 * c * g.ldb + k0) * E;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          u32x4 v = {0, 0, 0, 0};
          if (nc > 16 * c) {
            if constexpr (kPartial) v = k_chunk<E>(p + 16 * h, left - h * (16 / E));
            else v = load16(p + 16 * h);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) x.r[8 * c + 4 * h + i] = v[i];
        }
      }
    }
  };
  // fragment of columns tile c, instruction f
  auto frag_b = [&](const Raw& x, int c, int f) {
    Frag o;
    if constexpr (B_MN) {
      const uint32_t sel = c ? 0x07060302u : 0x05040100u;   // high or low halves of two k-rows
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __builtin_amdgcn_perm(x.r[2 * e + 1], x.r[2 * e], sel);
    } else if constexpr (E == 2) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = x.r[8 * c + 4 * f + e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = x.r[8 * c + e];
    }
    return o;
  };
  // A's fragment of row tile i, instruction f of a step: K in the same order as B's
  auto frag_a = [&](int step, int i, int f, auto partial) {
    constexpr bool kPartial = decltype(partial)::value;
    const int row = 16 * i + li, k = step * KS + kl + (E == 2 ? 8 * f : 0), left = K - k;
    Frag o = {};
    if (row < g.M) {
      if constexpr (A_MN) {
        o = k_gather((const uint16_t*)pa + (int64_t)k * g.lda + row, g.lda, kPartial ? left : 8);
      } else {
        const uint8_t* p = pa + ((int64_t)row * g.lda + k) * E;
        if constexpr (E == 2) {
          o = kPartial ? k_chunk<E>(p, left) : load16(p);
        } else {
          const u32x4 a = kPartial ? k_chunk<E>(p, left) : load16(p);
          const u32x4 b = kPartial ? k_chunk<E>(p + 16, left - 16) : load16(p + 16);
          o = Frag{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
        }
      }
    }
    return o;
  };

  f32x4 acc[MT][NI];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int c = 0; c < NI; ++c) acc[i][c] = f32x4{};
  auto multiply = [&](const Raw& x, const Frag (&a)[MT][NF]) {
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int c = 0; c < NI; ++c) {
        const Frag b = frag_b(x, c, f);
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i][c] = mfma16t<DT>(b, a[i][f], acc[i][c]);
      }
  };
  using T_ = std::true_type;
  using F_ = std::false_type;
  int s = wave;
  // `n` of this wave's steps at once: every load is on its way before the first wait
  auto batch = [&](auto n, auto partial) {
    constexpr int NB = decltype(n)::value;
    Raw x[NB];
    Frag a[NB][MT][NF];
#pragma unroll
    for (int u = 0; u < NB; ++u) load_b(s + u * W, partial, x[u]);
#pragma unroll
    for (int u = 0; u < NB; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int f = 0; f < NF; ++f) a[u][i][f] = frag_a(s + u * W, i, f, partial);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < NB; ++u) multiply(x[u], a[u]);
    s += NB * W;
  };
  while (s + (U - 1) * W < full) batch(std::integral_constant<int, U>{}, F_{});
  if (s + W < full) batch(std::integral_constant<int, 2>{}, F_{});
  if (s < full) batch(std::integral_constant<int, 1>{}, F_{});
  if (s < T) batch(std::integral_constant<int, 1>{}, T_{});   // the partial step, if it is this wave's

  // lane: row 16i + li, columns 4·lg + r of tile c (column 2j + c of the workgroup if B_MN)
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int c = 0; c < NI; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        red[wave][16 * i + li][B_MN ? 2 * (4 * lg + r) + c : 16 * c + 4 * lg + r] = acc[i][c][r];
  __syncthreads();
  auto sum = [&](int row, int n) {
    float v = red[0][row][n];
    if (W == 16) {
#pragma unroll
      for (int w = 1; w < 16; ++w) v += red[w][row][n];
    } else {
      for (int w = 1; w < W; ++w) v += red[w][row][n];
    }
    return v;
  };
  for (int o = (int)threadIdx.x; o < MT * 16 * CN; o += (int)blockDim.x) {
    const int row = o / CN, col_o = n0 + o % CN;
    if (row >= g.M || col_o >= n1) continue;
    const float v = sum(row, o % CN);
    if (g.splits > 1) {
      g.part[((int64_t)split * g.M + row) * g.part_ld + col_o] = v;
    } else {
      if (o != (int)threadIdx.x) ep_one(g, row, col_o, pre);
      ep_finish1(g, row, col_o, pre, v);
    }
  }
}

template <bool A_MN, bool B_MN, int DT>
hipError_t go(const EpArgs& g, int waves, hipStream_t s) {
  const dim3 grid((unsigned)((((int64_t)g.N + g.cn - 1) / g.cn) * g.splits)), block(64 * (unsigned)waves);
  constexpr int N1 = B_MN ? 2 : 1;
  const bool wide = B_MN || g.cn == 32;
  if (g.M <= 16) {
    if (wide) hipLaunchKernelGGL((gemm_ep_tokens<A_MN, B_MN, DT, 1, 2>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((gemm_ep_tokens<A_MN, B_MN, DT, 1, N1>), grid, block, 0, s, g);
  } else {
    if (wide) hipLaunchKernelGGL((gemm_ep_tokens<A_MN, B_MN, DT, 2, 2>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((gemm_ep_tokens<A_MN, B_MN, DT, 2, N1>), grid, block, 0, s, g);
  }
  return hipGetLastError();
}
template <int DT>
hipError_t go16(const EpArgs& g, int ta, int tb, int waves, hipStream_t s) {
  if (ta) return tb ? go<true, false, DT>(g, waves, s) : go<true, true, DT>(g, waves, s);
  return tb ? go<false, false, DT>(g, waves, s) : go<false, true, DT>(g, waves, s);
}

}  // namespace

hipError_t launch_ep_tokens(const EpArgs& g, int trans_a, int trans_b, int a_dtype, int b_dtype, int waves,
                            hipStream_t s) {
  if (a_dtype == TG_F16) return go16<TG_F16>(g, trans_a, trans_b, waves, s);
  if (a_dtype == TG_BF16) return go16<TG_BF16>(g, trans_a, trans_b, waves, s);
  const bool a5 = a_dtype == TG_FP8_E5M2, b5 = b_dtype == TG_FP8_E5M2;
  if (a5 && b5) return go<false, false, fp8_code(1, 1)>(g, waves, s);
  if (a5) return go<false, false, fp8_code(1, 0)>(g, waves, s);
  if (b5) return go<false, false, fp8_code(0, 1)>(g, waves, s);
  return go<false, false, fp8_code(0, 0)>(g, waves, s);
}

}  // namespace tg
