// Matrix product with an epilogue: launch arguments and the epilogue's device functions.
//
//   P = A·B (fp32 sums)   Z = row_scale[m]·col_scale[n]·P + bias[n]   D = act(Z) + residual
//
// Every kernel that finishes an output element (the block kernels, the token kernels and the join
// of a split sum) goes through ep_finish, so all of them round once: Z and D are each
// rounded to d_dtype from the fp32 value.  Internal header.
#pragma once

#include <hip/hip_runtime.h>

#include "tg_internal.h"

namespace tg {

struct EpArgs {
  const uint8_t* A;
  const uint8_t* B;
  uint8_t* D;
  int64_t lda, ldb, ldd;       // elements
  int32_t M, N, K;
  int32_t tiles_m, tiles_n;
  int32_t splits, k_per_split; // the sum over K in `splits` parts of k_per_split (the last one shorter)
  float* part;                 // splits > 1: fp32 sums [splits][M][part_ld]
  int64_t part_ld;             // N rounded up to 8: rows stay 32-byte aligned
  const uint8_t* bias;
  const uint8_t* res;
  uint8_t* Z;
  const float* rs;
  const float* cs;
  int64_t ldr, ldz;
  int32_t bias_t, d_t, act;    // tg_dtype, tg_dtype, tg_act
};

// Kernel families of tile_gemm_ep (tg_ep_plan.kernel).
hipError_t launch_ep_block(const EpArgs& g, int trans_a, int trans_b, int a_dtype, int b_dtype, int bs,
                           bool staged, hipStream_t s);
hipError_t launch_ep_join(const EpArgs& g, hipStream_t s);

// dZ = dY·act'(Z) ([M][N] packed, may be NULL) and column sums [groups][N] (may be NULL).
struct ActGradArgs {
  const uint8_t* dY;
  const uint8_t* Z;
  uint8_t* dZ;
  float* sums;
  int64_t ldy, ldz;
  int32_t M, N, rows_per;   // rows per group
  int32_t t, act;
};
hipError_t launch_act_grad(const ActGradArgs& a, int groups, hipStream_t s);
// out[n] = sum_g part[g][n]
hipError_t launch_sum_rows(const float* part, int64_t G, int64_t N, float* out, hipStream_t s);

// one orientation per translation unit (ep_gemm_*.hip)
hipError_t launch_ep_kk(const EpArgs& g, int dtype, int bs, bool staged, hipStream_t s);
hipError_t launch_ep_km(const EpArgs& g, int dtype, int bs, bool staged, hipStream_t s);
hipError_t launch_ep_mk(const EpArgs& g, int dtype, int bs, bool staged, hipStream_t s);
hipError_t launch_ep_mm(const EpArgs& g, int dtype, int bs, bool staged, hipStream_t s);
hipError_t launch_ep_fp8(const EpArgs& g, int a_dtype, int b_dtype, int bs, bool staged, hipStream_t s);

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
__device__ __forceinline__ void store16(void* p, ep_u32x4 v) { ((Bytes16*)p)->v = v; }

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
// n >= 1 valid elements of 8
__device__ __forceinline__ void ep_get8(const uint8_t* p, int t, int64_t i, int n, float (&v)[8]) {
  if (n >= 8) {
    if (t == TG_F32) {
      const ep_u32x4 a = load16(p + 4 * i), b = load16(p + 4 * i + 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = __builtin_bit_cast(float, (uint32_t)a[e]);
        v[4 + e] = __builtin_bit_cast(float, (uint32_t)b[e]);
      }
    } else {
      const ep_u32x4 a = load16(p + 2 * i);
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
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < n ? ep_get(p, t, i + e) : 0.0f;
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
__device__ __forceinline__ void ep_put8(uint8_t* p, int t, int64_t i, int n, const float (&v)[8]) {
  if (n >= 8) {
    if (t == TG_F32) {
      ep_u32x4 a, b;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = __builtin_bit_cast(uint32_t, v[e]);
        b[e] = __builtin_bit_cast(uint32_t, v[4 + e]);
      }
      store16(p + 4 * i, a);
      store16(p + 4 * i + 16, b);
    } else {
      store16(p + 2 * i, ep_pack8(t, v));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) ep_put(p, t, i + e, v[e]);
  }
}

// ---- activations ------------------------------------------------------------------------------
// sigmoid(x) = 1/(1 + e^-x): for x -> -inf e^-x overflows to +inf and the quotient is 0.
__device__ __forceinline__ float ep_sigmoid(float x) { return 1.0f / (1.0f + __expf(-x)); }

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2/pi)
constexpr float kGeluA = 0.044715f;

// 0.5 z (1 + tanh u) = z·sigmoid(2u): no difference of near-equal numbers for negative z.
// gelu = z·Phi(z) with Phi from erfc, for the same reason.
__device__ __forceinline__ float ep_act(float z, int act) {
  switch (act) {
    case TG_ACT_RELU: return z > 0.0f || z != z ? z : 0.0f;
    case TG_ACT_GELU: return 0.5f * z * erfcf(-0.70710678118654752f * z);
    case TG_ACT_GELU_TANH: return z * ep_sigmoid(2.0f * kGeluC * (z + kGeluA * z * z * z));
    case TG_ACT_SILU: return z * ep_sigmoid(z);
    default: return z;
  }
}
// Derivatives.  The argument is clamped where the derivative has reached 0 or 1 to below half
// a unit of fp32, so that z² and z³ of large finite z cannot make 0·inf; NaN passes through.
__device__ __forceinline__ float ep_act_grad(float z, int act) {
  const float c = z != z ? z : fminf(fmaxf(z, -100.0f), 100.0f);
  switch (act) {
    case TG_ACT_RELU: return z > 0.0f ? 1.0f : z != z ? z : 0.0f;
    case TG_ACT_GELU:
      return 0.5f * erfcf(-0.70710678118654752f * c) + c * 0.3989422804014327f * __expf(-0.5f * c * c);
    case TG_ACT_GELU_TANH: {
      const float s = ep_sigmoid(2.0f * kGeluC * (c + kGeluA * c * c * c));
      return s + c * s * (1.0f - s) * 2.0f * kGeluC * (1.0f + 3.0f * kGeluA * c * c);
    }
    case TG_ACT_SILU: {
      const float s = ep_sigmoid(c);
      return s * (1.0f + c * (1.0f - s));
    }
    default: return 1.0f;
  }
}

// ---- the epilogue of 8 consecutive columns -----------------------------------------------------
struct EpCols {   // per-column values of the lane's 8 columns, loaded once
  float bias[8], cs[8];
};
__device__ __forceinline__ void ep_cols(const EpArgs& g, int col, EpCols& c) {
  const int n = g.N - col;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    c.bias[e] = 0.0f;
    c.cs[e] = 1.0f;
  }
  if (n <= 0) return;
  if (g.bias) ep_get8(g.bias, g.bias_t, col, n, c.bias);
  if (g.cs) ep_get8((const uint8_t*)g.cs, TG_F32, col, n, c.cs);
}
// v: the sums P of row `row`, columns col .. col+7 (row < M, col < N)
__device__ __forceinline__ void ep_finish8(const EpArgs& g, int row, int col, const EpCols& c,
                                           float (&v)[8]) {
  const int n = g.N - col;
  if (g.rs) {
    const float r = g.rs[row];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= r;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = v[e] * c.cs[e] + c.bias[e];
  if (g.Z) ep_put8(g.Z, g.d_t, (int64_t)row * g.ldz + col, n, v);
  if (g.act != TG_ACT_NONE) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = ep_act(v[e], g.act);
  }
  if (g.res) {
    float r[8];
    ep_get8(g.res, g.d_t, (int64_t)row * g.ldr + col, n, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += r[e];
  }
  ep_put8(g.D, g.d_t, (int64_t)row * g.ldd + col, n, v);
}
// one element
__device__ __forceinline__ void ep_finish1(const EpArgs& g, int row, int col, float p) {
  if (g.rs) p *= g.rs[row];
  if (g.cs) p *= g.cs[col];
  if (g.bias) p += ep_get(g.bias, g.bias_t, col);
  if (g.Z) ep_put(g.Z, g.d_t, (int64_t)row * g.ldz + col, p);
  p = ep_act(p, g.act);
  if (g.res) p += ep_get(g.res, g.d_t, (int64_t)row * g.ldr + col);
  ep_put(g.D, g.d_t, (int64_t)row * g.ldd + col, p);
}

}  // namespace
#endif

}  // namespace tg
