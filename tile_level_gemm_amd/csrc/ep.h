// Matrix product with an epilogue: launch arguments and the epilogue's device functions.
//
//   P = A·B (fp32 sums; int8 operands: exact 32-bit integers, then fp32)   Z = row_scale[m]·col_scale[n]·P + bias[n]   D = act(Z) + residual
//
// Gated: B has 2N columns, the gate's and the up projection's, Z = [G | U] has them too, and D = act(G)·U
// has N.
//
// Every kernel that finishes an output element (the block kernels, the token kernels and the join
// of a split sum) goes through ep_finish8, its 16-bit form or ep_finish1, or the gated_* ones, so all of them
// round once: Z and D are each rounded to d_dtype from the fp32 value.  Internal header.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "tg_internal.h"

namespace tg {

struct EpArgs {
  const uint8_t* A;
  const uint8_t* B;
  uint8_t* D;
  int64_t lda, ldb, ldd;       // elements
  int32_t M, N, K;             // N: columns of D
  int32_t tiles_m, tiles_n;
  int32_t waves, cn;           // few rows: waves and columns of a workgroup
  int32_t ring;                // direct blocks: four stages in flight (128 and 64 wide)
  int32_t splits, k_per_split; // the sum over K in `splits` parts of k_per_split (the last one shorter)
  float* part;                 // splits > 1: fp32 (or 32-bit integer) sums [splits][M][part_ld]
  int64_t part_ld;             // N rounded up to 8: rows stay 32-byte aligned; gated: twice that, U in the second half
  const uint8_t* bias;
  const uint8_t* res;
  uint8_t* Z;
  const float* rs;
  const float* cs;
  int64_t ldr, ldz;
  int32_t bias_t, d_t, act;    // tg_dtype, tg_dtype, tg_act
  int32_t ints;                // parts hold integers
};

// Kernel families of tile_gemm_ep (tg_ep_plan.kernel).
struct EpKernel {   // block kernels: block size 64 or 128 (staged, ring), 128 or 256 (direct)
  int bs;
  bool staged, ring;
  bool fine = false;   // 256-wide blocks of 16-bit products that are not gated: the 16-row matrix instructions
};
hipError_t launch_ep_block(const EpArgs& g, int trans_a, int trans_b, int a_dtype, int b_dtype,
                           const EpKernel& k, hipStream_t s);
// M <= kTokenRows; `waves` (1 .. 16) waves share K
constexpr int64_t kTokenRows = 32;
hipError_t launch_ep_tokens(const EpArgs& g, int trans_a, int trans_b, int a_dtype, int b_dtype, int waves,
                            hipStream_t s);
hipError_t launch_ep_join(const EpArgs& g, bool gated, hipStream_t s);
// A [M,K]; B [2N,K] (trans_b) or [K,2N], the latter for 16-bit operands
hipError_t launch_gated_block(const EpArgs& g, int trans_b, int a_dtype, int b_dtype, const EpKernel& k, hipStream_t s);
// M <= kTokenRows, B [2N,K]
hipError_t launch_gated_tokens(const EpArgs& g, int a_dtype, int b_dtype, int waves, hipStream_t s);

// dZ = dY·act'(Z) ([M][N] packed, may be NULL) and column sums [groups][N] (may be NULL).  With scales the
// sums are of that, and dZ receives row_scale·col_scale·dY·act'(Z).
struct ActGradArgs {
  const uint8_t* dY;
  const uint8_t* Z;
  uint8_t* dZ;
  float* sums;
  const float* rs;   // row and column scales, or NULL
  const float* cs;
  int64_t ldy, ldz;
  int32_t M, N, rows_per;   // rows per group
  int32_t t, act;
};
hipError_t launch_act_grad(const ActGradArgs& a, int groups, hipStream_t s);
// The same of D = act(G)·U, Z = [G | U] and dZ [M][2N] = [dY·U·act'(G) | dY·act(G)], column scales, sums [groups][2N];
// N: columns of D.
hipError_t launch_gated_grad(const ActGradArgs& a, int groups, hipStream_t s);
// out[n] = sum_g part[g][n]; columns from `split` on go to rest[n - split]
hipError_t launch_sum_rows(const float* part, int64_t G, int64_t N, float* out, hipStream_t s,
                           float* rest = nullptr, int64_t split = INT64_MAX);

// one orientation per translation unit (ep_gemm_*.hip)
hipError_t launch_ep_kk(const EpArgs& g, int dtype, const EpKernel& k, hipStream_t s);
hipError_t launch_ep_km(const EpArgs& g, int dtype, const EpKernel& k, hipStream_t s);
hipError_t launch_ep_mk(const EpArgs& g, int dtype, const EpKernel& k, hipStream_t s);
hipError_t launch_ep_mm(const EpArgs& g, int dtype, const EpKernel& k, hipStream_t s);
hipError_t launch_ep_fp8(const EpArgs& g, int a_dtype, int b_dtype, const EpKernel& k, hipStream_t s);
hipError_t launch_ep_i8(const EpArgs& g, const EpKernel& k, hipStream_t s);
hipError_t launch_gated_8(const EpArgs& g, int a_dtype, int b_dtype, const EpKernel& k, hipStream_t s);

#ifdef __HIP__
namespace {

// ---- loads and stores of up to W consecutive elements -------------------------------------
// Rows may start at any element (odd leading dimensions), so the vector forms state the
// element's own alignment: global memory takes 16-byte accesses at 2-byte addresses.
typedef __attribute__((ext_vector_type(4))) uint32_t ep_u32x4;
typedef __attribute__((ext_vector_type(2))) __bf16 ep_bf16x2;
typedef __attribute__((ext_vector_type(2))) _Float16 ep_f16x2;
typedef __attribute__((ext_vector_type(2))) float ep_f32x2;

struct __attribute__((packed, aligned(1))) Bytes16 { ep_u32x4 v; };
__device__ __forceinline__ ep_u32x4 load16(const void* p) { return ((const Bytes16*)p)->v; }
typedef ep_u32x4 __attribute__((aligned(1))) ep_u32x4_any;
// NT: a result that nothing here reads again streams past the L2, where the operands stay
template <bool NT = false>
__device__ __forceinline__ void store16(void* p, ep_u32x4 v) {
  if constexpr (NT) __builtin_nontemporal_store(v, (ep_u32x4_any*)p);
  else ((Bytes16*)p)->v = v;
}

__device__ __forceinline__ float ep_get(const uint8_t* p, int t, int64_t i) {
  if (t == TG_F32) return ((const float*)p)[i];
  if (t == TG_BF16) return (float)((const __bf16*)p)[i];
  return (float)((const _Float16*)p)[i];
}
__device__ __forceinline__ void ep_put(uint8_t* p, int t, int64_t i, float v) {
  if (t == TG_F32) ((float*)p)[i] = v;
  else if (t == TG_BF16) ((__bf16*)p)[i] = (__bf16)v;
  else ((_Float16*)p)[i] = (_Float16)v;
}
// 8 16-bit elements
__device__ __forceinline__ void ep_unpack8(int t, ep_u32x4 a, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w = a[e];
    if (t == TG_BF16) {
      v[2 * e] = __builtin_bit_cast(float, w << 16);
      v[2 * e + 1] = __builtin_bit_cast(float, w & 0xffff0000u);
    } else {
      const ep_f16x2 h = __builtin_bit_cast(ep_f16x2, w);
      v[2 * e] = (float)h[0];
      v[2 * e + 1] = (float)h[1];
    }
  }
}
// n >= 1 valid elements of 8, zeros behind them.  At a row's end the last element is loaded again where
// there is none, so that the eight loads wait together.
__device__ __forceinline__ ep_u32x4 ep_load8_16(const uint8_t* p, int64_t i, int n) {
  if (n >= 8) return load16(p + 2 * i);
  uint16_t u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) u[e] = ((const uint16_t*)p)[i + min(e, n - 1)];
  ep_u32x4 w;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w[e] = (2 * e < n ? (uint32_t)u[2 * e] : 0u) | (2 * e + 1 < n ? (uint32_t)u[2 * e + 1] << 16 : 0u);
  return w;
}
__device__ __forceinline__ void ep_get8(const uint8_t* p, int t, int64_t i, int n, float (&v)[8]) {
  if (t != TG_F32) {
    ep_unpack8(t, ep_load8_16(p, i, n), v);
  } else if (n >= 8) {
    const ep_u32x4 a = load16(p + 4 * i), b = load16(p + 4 * i + 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = __builtin_bit_cast(float, (uint32_t)a[e]);
      v[4 + e] = __builtin_bit_cast(float, (uint32_t)b[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = ((const float*)p)[i + min(e, n - 1)];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < n ? v[e] : 0.0f;
  }
}
__device__ __forceinline__ ep_u32x4 ep_pack8(int t, const float (&v)[8]) {
  ep_u32x4 o;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const ep_f32x2 f = {v[2 * e], v[2 * e + 1]};
    if (t == TG_BF16) o[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, ep_bf16x2));
    else o[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, ep_f16x2));
  }
  return o;
}
template <bool NT = false>
__device__ __forceinline__ void ep_store8_16(uint8_t* p, int64_t i, int n, ep_u32x4 w) {
  if (n >= 8) {
    store16<NT>(p + 2 * i, w);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) ((uint16_t*)p)[i + e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
  }
}
__device__ __forceinline__ void ep_put8(uint8_t* p, int t, int64_t i, int n, const float (&v)[8]) {
  if (t != TG_F32) {
    ep_store8_16(p, i, n, ep_pack8(t, v));
  } else if (n >= 8) {
    ep_u32x4 a, b;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = __builtin_bit_cast(uint32_t, v[e]);
      b[e] = __builtin_bit_cast(uint32_t, v[4 + e]);
    }
    store16(p + 4 * i, a);
    store16(p + 4 * i + 16, b);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) ((float*)p)[i + e] = v[e];
  }
}

// ---- activations ------------------------------------------------------------------------------
// The sigmoid and the tail of the normal distribution take the unit's own reciprocal (1 ulp) and
// exp2: an IEEE quotient costs ten instructions more per element, and the epilogue of a 256-wide
// block does not overlap its products.

// 1/(1 + 2^x): for x -> +inf 2^x is +inf and the quotient 0.
__device__ __forceinline__ float ep_inv1p2(float x) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x)); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2/pi)
constexpr float kGeluA = 0.044715f;
constexpr float kGeluE = -2.0f * kGeluC * kLog2e;

// sigmoid(x) and sigmoid(2u), 2u = 2c(z + a z^3)
__device__ __forceinline__ float ep_sigmoid(float x) { return ep_inv1p2(-kLog2e * x); }
__device__ __forceinline__ float ep_gelu_sigmoid(float z) { return ep_inv1p2(kGeluE * z * (1.0f + kGeluA * z * z)); }

// 0.5·erfc(-z/sqrt(2)) = Phi(z).  erfc by the Chebyshev fit of Press et al., Numerical Recipes
// (erfcc): t·exp(-x² + p(t)), t = 1/(1 + x/2), within 1.2e-7 of the value for every x >= 0; so
// small tails keep their relative accuracy.
__device__ __forceinline__ float ep_phi(float z) {
  const float x = fabsf(z) * 0.70710678118654752f;
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.5f * x);
  float p = 0.17087277f;
  p = fmaf(p, t, -0.82215223f);
  p = fmaf(p, t, 1.48851587f);
  p = fmaf(p, t, -1.13520398f);
  p = fmaf(p, t, 0.27886807f);
  p = fmaf(p, t, -0.18628806f);
  p = fmaf(p, t, 0.09678418f);
  p = fmaf(p, t, 0.37409196f);
  p = fmaf(p, t, 1.00002368f);
  p = fmaf(p, t, -1.26551223f);
  const float q = 0.5f * t * __builtin_amdgcn_exp2f(kLog2e * (p - 0.5f * z * z));
  return z > 0.0f ? 1.0f - q : q;
}

// 0.5 z (1 + tanh u) = z·sigmoid(2u): no difference of near-equal numbers for negative z.
// gelu = z·Phi(z) with Phi from erfc, for the same reason.
template <int ACT>
__device__ __forceinline__ float ep_act(float z) {
  if constexpr (ACT == TG_ACT_RELU) return z > 0.0f || z != z ? z : 0.0f;
  else if constexpr (ACT == TG_ACT_GELU) return z * ep_phi(z);
  else if constexpr (ACT == TG_ACT_GELU_TANH) return z * ep_gelu_sigmoid(z);
  else if constexpr (ACT == TG_ACT_SILU) return z * ep_sigmoid(z);
  else return z;
}
// Derivatives.  The argument is clamped where the derivative has reached 0 or 1 to below half
// a unit of fp32, so that z² and z³ of large finite z cannot make 0·inf; NaN passes through.
template <int ACT>
__device__ __forceinline__ float ep_act_grad(float z) {
  const float c = z != z ? z : fminf(fmaxf(z, -100.0f), 100.0f);
  if constexpr (ACT == TG_ACT_RELU) {
    return z > 0.0f ? 1.0f : z != z ? z : 0.0f;
  } else if constexpr (ACT == TG_ACT_GELU) {
    return ep_phi(c) + c * 0.3989422804014327f * __builtin_amdgcn_exp2f(-0.5f * kLog2e * c * c);
  } else if constexpr (ACT == TG_ACT_GELU_TANH) {
    const float s = ep_gelu_sigmoid(c);
    return s + c * s * (1.0f - s) * 2.0f * kGeluC * (1.0f + 3.0f * kGeluA * c * c);
  } else if constexpr (ACT == TG_ACT_SILU) {
    const float s = ep_sigmoid(c);
    return s * (1.0f + c * (1.0f - s));
  } else {
    return 1.0f;
  }
}
// f(activation) with the activation as a compile-time constant
template <class F>
__device__ __forceinline__ void ep_with_act(int act, F f) {
  switch (act) {
    case TG_ACT_RELU: f(std::integral_constant<int, TG_ACT_RELU>{}); break;
    case TG_ACT_GELU: f(std::integral_constant<int, TG_ACT_GELU>{}); break;
    case TG_ACT_GELU_TANH: f(std::integral_constant<int, TG_ACT_GELU_TANH>{}); break;
    case TG_ACT_SILU: f(std::integral_constant<int, TG_ACT_SILU>{}); break;
    default: f(std::integral_constant<int, TG_ACT_NONE>{}); break;
  }
}

// ---- the epilogue of 8 consecutive columns -----------------------------------------------------
struct EpCols {   // per-column values of the lane's 8 columns, loaded once
  float bias[8], cs[8];
};
// first: column 0 of those that the lane's are counted from (gated: N for the up projection's)
__device__ __forceinline__ void ep_cols(const EpArgs& g, int col, EpCols& c, int first = 0) {
  const int n = g.N - col;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    c.bias[e] = 0.0f;
    c.cs[e] = 1.0f;
  }
  if (n <= 0) return;
  if (g.bias) ep_get8(g.bias, g.bias_t, (int64_t)first + col, n, c.bias);
  if (g.cs) ep_get8((const uint8_t*)g.cs, TG_F32, (int64_t)first + col, n, c.cs);
}
// v: the sums P of row `row`, columns col .. col+7 (row < M, col < N); any type, any number of
// columns left.
__device__ __forceinline__ void ep_finish8(const EpArgs& g, int row, int col, const EpCols& c, float (&v)[8]) {
  const int n = g.N - col;
  const float rs = g.rs ? g.rs[row] : 1.0f;
  float r[8] = {};
  if (g.res) ep_get8(g.res, g.d_t, (int64_t)row * g.ldr + col, n, r);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = v[e] * rs * c.cs[e] + c.bias[e];
  if (g.Z) ep_put8(g.Z, g.d_t, (int64_t)row * g.ldz + col, n, v);
  ep_with_act(g.act, [&](auto act) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = ep_act<decltype(act)::value>(v[e]);
  });
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] += r[e];
  ep_put8(g.D, g.d_t, (int64_t)row * g.ldd + col, n, v);
}
// one element: what its epilogue reads, and the finish
struct EpOne {
  float rs, cs, bias, res;
};
__device__ __forceinline__ void ep_one(const EpArgs& g, int row, int col, EpOne& x) {
  x.rs = g.rs ? g.rs[row] : 1.0f;
  x.cs = g.cs ? g.cs[col] : 1.0f;
  x.bias = g.bias ? ep_get(g.bias, g.bias_t, col) : 0.0f;
  x.res = g.res ? ep_get(g.res, g.d_t, (int64_t)row * g.ldr + col) : 0.0f;
}
__device__ __forceinline__ void ep_finish1(const EpArgs& g, int row, int col, const EpOne& x, float p) {
  p = p * x.rs * x.cs + x.bias;
  if (g.Z) ep_put(g.Z, g.d_t, (int64_t)row * g.ldz + col, p);
  ep_with_act(g.act, [&](auto act) { p = ep_act<decltype(act)::value>(p); });
  ep_put(g.D, g.d_t, (int64_t)row * g.ldd + col, p + x.res);
}
// 8 columns of 16-bit results, in two halves: what a row needs besides its sums is loaded for several
// rows ahead of their stores (the residual may be D, so the compiler would not move its load above a
// store).
struct EpRow {
  float rs;
  ep_u32x4 res;
};
__device__ __forceinline__ void ep_row(const EpArgs& g, int row, int col, EpRow& x) {
  x.rs = g.rs ? g.rs[row] : 1.0f;
  if (g.res) x.res = ep_load8_16(g.res, (int64_t)row * g.ldr + col, g.N - col);
}
template <int ACT>
__device__ __forceinline__ void ep_finish8_16(const EpArgs& g, int row, int col, const EpCols& c, const EpRow& x,
                                                float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = v[e] * x.rs * c.cs[e] + c.bias[e];
  if (g.Z) ep_store8_16<true>(g.Z, (int64_t)row * g.ldz + col, g.N - col, ep_pack8(g.d_t, v));
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = ep_act<ACT>(v[e]);
  if (g.res) {
    float r[8];
    ep_unpack8(g.d_t, x.res, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += r[e];
  }
  ep_store8_16<true>(g.D, (int64_t)row * g.ldd + col, g.N - col, ep_pack8(g.d_t, v));
}

// ---- gated: 8 consecutive columns of the gate and of the up projection ---------------------------
struct GatedCols {
  EpCols gate, up;
};
__device__ __forceinline__ void gated_cols(const EpArgs& g, int col, GatedCols& c) {
  ep_cols(g, col, c.gate);
  ep_cols(g, col, c.up, g.N);
}
__device__ __forceinline__ void gated_z(const EpArgs& g, int row, const GatedCols& c, float (&v)[8], float (&u)[8]) {
  const float rs = g.rs ? g.rs[row] : 1.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[e] = v[e] * rs * c.gate.cs[e] + c.gate.bias[e];
    u[e] = u[e] * rs * c.up.cs[e] + c.up.bias[e];
  }
}
// v, u: the sums of both projections; any type, any number of columns left
__device__ __forceinline__ void gated_finish8(const EpArgs& g, int row, int col, const GatedCols& c, float (&v)[8],
                                              float (&u)[8]) {
  const int n = g.N - col;
  gated_z(g, row, c, v, u);
  if (g.Z) {
    ep_put8(g.Z, g.d_t, (int64_t)row * g.ldz + col, n, v);
    ep_put8(g.Z, g.d_t, (int64_t)row * g.ldz + g.N + col, n, u);
  }
  ep_with_act(g.act, [&](auto act) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = ep_act<decltype(act)::value>(v[e]) * u[e];
  });
  ep_put8(g.D, g.d_t, (int64_t)row * g.ldd + col, n, v);
}
template <int ACT>
__device__ __forceinline__ void gated_finish8_16(const EpArgs& g, int row, int col, const GatedCols& c, float (&v)[8],
                                                 float (&u)[8]) {
  const int n = g.N - col;
  gated_z(g, row, c, v, u);
  if (g.Z) {
    ep_store8_16<true>(g.Z, (int64_t)row * g.ldz + col, n, ep_pack8(g.d_t, v));
    ep_store8_16<true>(g.Z, (int64_t)row * g.ldz + g.N + col, n, ep_pack8(g.d_t, u));
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = ep_act<ACT>(v[e]) * u[e];
  ep_store8_16<true>(g.D, (int64_t)row * g.ldd + col, n, ep_pack8(g.d_t, v));
}
// one element
struct GatedOne {
  float rs, cs[2], bias[2];
};
__device__ __forceinline__ void gated_one(const EpArgs& g, int row, int col, GatedOne& x) {
  x.rs = g.rs ? g.rs[row] : 1.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t at = (int64_t)h * g.N + col;
    x.cs[h] = g.cs ? g.cs[at] : 1.0f;
    x.bias[h] = g.bias ? ep_get(g.bias, g.bias_t, at) : 0.0f;
  }
}
__device__ __forceinline__ void gated_finish1(const EpArgs& g, int row, int col, const GatedOne& x, float v, float u) {
  v = v * x.rs * x.cs[0] + x.bias[0];
  u = u * x.rs * x.cs[1] + x.bias[1];
  if (g.Z) {
    ep_put(g.Z, g.d_t, (int64_t)row * g.ldz + col, v);
    ep_put(g.Z, g.d_t, (int64_t)row * g.ldz + g.N + col, u);
  }
  ep_with_act(g.act, [&](auto act) { v = ep_act<decltype(act)::value>(v); });
  ep_put(g.D, g.d_t, (int64_t)row * g.ldd + col, v * u);
}

}  // namespace
#endif

}  // namespace tg
