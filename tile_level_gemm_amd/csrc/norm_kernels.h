// Norms with the residual's addition and their backward passes, and the quantisation of rows: one set of
// kernels over NormKind.
//
//   H = X + R (rounded to X's type: it is the residual stream the next layer reads, and the
//   norm is taken of what that layer will see)
//   kRms     rstd = 1/sqrt(mean(H²) + eps)   xh = H·rstd   Y = xh·w
//   kLayer   m = mean(H)   rstd = 1/sqrt(mean((H − m)²) + eps)   xh = (H − m)·rstd   Y = xh·w + b
//   kRows    Y = X (8-bit results only)
//   8-bit Y: row scale s = max|Y|/qmax, or per 32 columns the smallest power of two s with
//   max|Y|/s <= qmax, so nothing saturates; Q = Y/s rounded once.  max|Y| is floored at 2^-100.
//   backward: g = dY·w, dX = rstd·(g − [kLayer: mean(g)] − xh·mean(g·xh)) + dH,
//   dw = Σ_rows dY·xh, kLayer: db = Σ_rows dY.
//
// All of it is bound by memory: one pass, the row kept in registers between the reduction and
// the result, NV chunks of 8 columns a thread.  Rows up to 1024 columns take one wave each and no
// barrier; longer ones a workgroup of as many waves as their chunks need (1003 x 2057: 5 waves of one
// chunk 5.4 us, 4 waves of two 6.2).  The sum of squares and max|H·w| (a row scale needs it:
// max|Y| = rstd·max|H·w|) travel in one reduction; a row whose max|H·w| is out of fp32's range
// (top_fits) takes a second one for max|Y| itself.  The layer norm reduces the sum, then the deviations from
// the mean and their squares (from registers; centre() has why), then max|Y| if a row scale needs it.
// Measured: 16384 x 8192 bf16 with residual to e4m3 blocks 163 us (5.8 TB/s of 944 MB); backward of
// 8192 x 8192 bf16 with dH 100 us and 4 for the sum of dw's shares (5.2 TB/s of 537 MB); one row of
// 4096 2.9 us, launch and latency.
// Rows whose length is not a multiple of 8 end in a chunk moved back to the row's last 8
// columns: every load is a whole vector, and the columns another chunk owns (`dup` of them) are left
// out of the sums.  Forward both owners store the same values; backward, where dX may be dH, a moved
// chunk stores its own columns only.
//
// Internal header: norm.hip has the instances of kRms, layer_norm.hip the others.
#pragma once

#include <algorithm>

#include "ep.h"
#include "norm.h"

namespace tg {
namespace {

constexpr float kAmaxFloor = 7.888609052210118e-31f;   // 2^-100

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}
// max that keeps NaN: a NaN in the row reaches its scale
__device__ __forceinline__ float nan_max(float a, float b) { return a != a || a > b ? a : b; }
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = nan_max(v, __shfl_xor(v, m));
  return v;
}

// Scale kind of a kernel's result: a tg_scale_kind, and with TG_SCALE_ROW integers apart from fp8.  Told apart by a
// branch on the type, the integers cost the RMS norm's fp8 rows 1 to 3 % (65536 x 136 bf16 33.1 -> 34.0 us).
constexpr int kRowInt = TG_SCALE_BLOCK + 1;
constexpr bool row_scaled(int sc) { return sc == TG_SCALE_ROW || sc == kRowInt; }

__device__ __forceinline__ float q_max(int t) { return t == TG_FP8_E4M3 ? 448.0f : 57344.0f; }

// 8 values to 8 bits (SC kRowInt: integers, else fp8 of type t); |v| <= qmax up to rounding, clamped there; NaN stays
// NaN, as an integer it is 0
template <int SC>
__device__ __forceinline__ uint2 quant8(const float (&v)[8], int t) {
  if constexpr (SC == kRowInt) {
    const float q = 127.0f;
    // v + 1.5·2^23 rounds v to the nearest integer, ties to even, and holds it in its low byte
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      b[e] = __builtin_bit_cast(uint32_t, (v[e] != v[e] ? 0.0f : fminf(fmaxf(v[e], -q), q)) + 12582912.0f);
    uint2 o;
    o.x = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u), __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), 0x05040100u);
    o.y = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[7], b[6], 0x0c0c0400u), __builtin_amdgcn_perm(b[5], b[4], 0x0c0c0400u), 0x05040100u);
    return o;
  }
  const float q = q_max(t);
  float c[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) c[e] = v[e] != v[e] ? v[e] : fminf(fmaxf(v[e], -q), q);
  int lo = 0, hi = 0;
  if (t == TG_FP8_E4M3) {
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], hi, true);
  } else {
    lo = __builtin_amdgcn_cvt_pk_bf8_f32(c[0], c[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_bf8_f32(c[2], c[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_bf8_f32(c[4], c[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_bf8_f32(c[6], c[7], hi, true);
  }
  return uint2{(uint32_t)lo, (uint32_t)hi};
}
typedef __attribute__((ext_vector_type(2))) uint32_t ep_u32x2;
struct __attribute__((packed, aligned(1))) Bytes8 { ep_u32x2 v; };

__device__ __forceinline__ void put_q8(uint8_t* p, int n, uint2 q) {
  if (n >= 8) {
    ((Bytes8*)p)->v = ep_u32x2{q.x, q.y};
  } else {
    for (int e = 0; e < n; ++e) p[e] = (uint8_t)((e < 4 ? q.x >> (8 * e) : q.y >> (8 * (e - 4))));
  }
}

// Exponent e of the smallest power of two with amax/2^e <= 1.75·2^top (448 = 1.75·2^8, 57344 =
// 1.75·2^15): the exponent of amax less `top`, one more when its fraction is above 1.75.
__device__ __forceinline__ int block_exp(float amax, int t) {
  const uint32_t b = __builtin_bit_cast(uint32_t, amax);
  return (int)((b + 0x1fffffu) >> 23) - 127 - (t == TG_FP8_E4M3 ? 8 : 15);
}

// Reduce (sum, max) over a row's threads; every thread gets the result.  WAVE: one wave, else the
// workgroup's waves, one slot of `red` each.
constexpr int kMaxWaves = 16;
template <bool WAVE>
__device__ __forceinline__ void row_reduce(float& s, float& m, bool want_max, float (*red)[2]) {
  s = wave_sum(s);
  if (want_max) m = wave_max(m);
  if constexpr (!WAVE) {
    const int w = (int)threadIdx.x >> 6, n = (int)blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      red[w][0] = s;
      red[w][1] = m;
    }
    __syncthreads();
    s = 0.0f;
    m = red[0][1];
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      s += red[i][0];
      if (want_max) m = nan_max(m, red[i][1]);
    }
  }
}

// The same for the layer norm and the quantised rows, without a trip through LDS for every step: within 16 lanes
// by rotations on the way into the addition, then lane rows exchanged, then one LDS read of the waves' values by
// 16 lanes each (bf16 layer norm gradients 8192 x 8192 119 us, 125 with row_reduce's shuffles; 16384 x 8192 to e4m3
// rows 171, 187).
template <int N>
__device__ __forceinline__ float lane_ror(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x120 + N, 0xf, 0xf, true));
}
struct Plus {
  __device__ __forceinline__ static float of(float a, float b) { return a + b; }
};
struct Most {
  __device__ __forceinline__ static float of(float a, float b) { return nan_max(a, b); }
};
template <class OP>
__device__ __forceinline__ float over_16(float v) {
  v = OP::of(v, lane_ror<8>(v));
  v = OP::of(v, lane_ror<4>(v));
  v = OP::of(v, lane_ror<2>(v));
  return OP::of(v, lane_ror<1>(v));
}
template <class OP>
__device__ __forceinline__ float over_wave(float v) {
  v = over_16<OP>(v);
  uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = OP::of(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
  u = __builtin_bit_cast(uint32_t, v);
  const auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return OP::of(__builtin_bit_cast(float, (uint32_t)b[0]), __builtin_bit_cast(float, (uint32_t)b[1]));
}
// S: of s; Q: of q, or void where there is none.  Maxima are of magnitudes: 0 at least.
template <bool WAVE, class S, class Q>
__device__ __forceinline__ void row_join(float& s, float& q, float (*red)[2]) {
  constexpr bool kBoth = !std::is_same<Q, void>::value;
  s = over_wave<S>(s);
  if constexpr (kBoth) q = over_wave<Q>(q);
  if constexpr (!WAVE) {
    const int w = (int)threadIdx.x >> 6, n = (int)blockDim.x >> 6, l = (int)threadIdx.x & 15;
    if ((threadIdx.x & 63) == 0) {
      red[w][0] = s;
      if constexpr (kBoth) red[w][1] = q;
    }
    __syncthreads();
    s = over_16<S>(l < n ? red[l][0] : 0.0f);
    if constexpr (kBoth) q = over_16<Q>(l < n ? red[l][1] : 0.0f);
  }
}

// The layer norm's centre and variance.  `mean` is the rounded quotient of a rounded sum, off by a few units of itself:
// in a row far from zero that is much beside its deviations, and in a row of one value it is all there is.  The
// deviations from it are nearly exact, so their mean (ds/n) says how far it is off, and their mean square less that
// one's is the variance about the true mean: 8192 fp32 values about 1e4 have Y within 1e-6, with the rounded mean alone
// 3.5e-4 off.  The reduction of the squares takes both sums (16384 x 8192 bf16 with residual 184 us, 183 without; to
// e4m3 rows 174, 170; 16384 x 4096 to e4m3 rows 103, 98).  Returns the variance; shift: what the mean lacks (0 where
// the row is not finite, whose mean and squares say so).
__device__ __forceinline__ float centre(float ss, float ds, float n, float& shift) {
  shift = ds / n;
  shift = fabsf(shift) < __builtin_inff() ? shift : 0.0f;
  const float v = ss / n;
  return v < __builtin_inff() ? fmaxf(fmaf(-shift, shift, v), 0.0f) : v;   // NaN and infinity stay
}

// Whether rstd·max|H·w| is max|Y|: the product with the weight has neither overflowed nor lost bits
// below the floor of max|Y| (NaN: no).
__device__ __forceinline__ bool top_fits(float top) { return top >= kAmaxFloor && top < __builtin_inff(); }
// Row scale of max|Y| >= the floor; NaN for a row with a NaN or an infinity.  For integers the product with
// 1/127 in fp32, which is what torch computes on the GPU for max / 127: a weight quantised there and one quantised here
// have the same codes.  By the quotient 4.4 % of 4096 rows of 8192 bf16 values had a scale one unit off, and 30 of the
// 33.5 million codes differed (half of a row's maximum is 63.5 steps, so the scale's last bit decides it).  The values
// that the codes stand for are as exact either way, 0.28863 steps off in the mean square: codes are rounded by the
// scale that is stored.
template <int SC>
__device__ __forceinline__ float row_scale(float amax, int t) {
  amax = nan_max(amax, kAmaxFloor);
  const float s = SC == kRowInt ? amax * (1.0f / 127.0f) : amax / q_max(t);
  return amax < __builtin_inff() ? s : __builtin_nanf("");
}
// y/s rounded to nearest for inv = 1/s rounded to nearest: Markstein's correction (IBM J. Res. Dev. 34,
// 1990) of the product.  The codes are then the quotient by the very scale that is stored; the product
// alone lands on the other side of a border once in some million codes.  Two operations an element
// (16384 x 8192 bf16 166 us; 164.7 without), where the quotient itself takes ten (172).  The correction
// of an exact quotient is -0 and leaves a zero its sign; the RMS norm's is +0, as its fp8 codes always were: both of
// its zeros have code 0.
template <int KIND>
__device__ __forceinline__ float quotient(float y, float s, float inv) {
  const float q = y * inv;
  return fmaf(KIND == kRms ? fmaf(-q, s, y) : -fmaf(q, s, -y), inv, q);
}

// SC: scale kind of the result
// WAVE: a wave per row, four rows a workgroup; else a workgroup per row.
template <int KIND, int DT, int NV, int SC, bool WAVE, int MAXT>
__global__ __launch_bounds__(MAXT) void norm_rows(NormArgs a) {
  // one for each reduction: no wave may still be reading where another writes
  __shared__ float red[KIND == kLayer ? 3 : 1][WAVE ? 1 : kMaxWaves][2];
  const int TPR = WAVE ? 64 : (int)blockDim.x;
  const int t = WAVE ? (int)threadIdx.x & 63 : (int)threadIdx.x;
  const int64_t row = WAVE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
  if (WAVE && row >= a.rows) return;
  const int cols = (int)a.cols;
  float h[NV][8], w[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) ep_get8(a.X, DT, row * a.ldx + min((j * TPR + t) * 8, cols - 8), 8, h[j]);
  if (KIND != kRows && a.R) {
    float r[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) ep_get8(a.R, DT, row * a.ldr + min((j * TPR + t) * 8, cols - 8), 8, r[j]);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = h[j][e] + r[j][e];
        if constexpr (DT == TG_BF16) h[j][e] = (float)(__bf16)x;
        else if constexpr (DT == TG_F16) h[j][e] = (float)(_Float16)x;
        else h[j][e] = x;
      }
  }
  if constexpr (KIND == kRms) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = min((j * TPR + t) * 8, cols - 8);
      if (a.w_t == TG_F32) ep_get8(a.W, TG_F32, col, 8, w[j]);
      else ep_get8(a.W, DT, col, 8, w[j]);
    }
  }
  constexpr bool EARLY = KIND == kLayer && NV == 1 && DT != TG_F32;
  ep_u32x4 rw = {0, 0, 0, 0}, rb = {0, 0, 0, 0};
  if (EARLY && a.w_t != TG_F32) {
    const int64_t col = min(t * 8, cols - 8);
    rw = load16(a.W + 2 * col);
    if (a.B) rb = load16(a.B + 2 * col);
  }
  float ss = 0.0f, ds = 0.0f, top = 0.0f, mean = 0.0f, back = 0.0f, rstd = 1.0f, none = 0.0f;
  if constexpr (KIND == kLayer) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int dup = (j * TPR + t) * 8 - (cols - 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) mean += e >= dup ? h[j][e] : 0.0f;
    }
    row_join<WAVE, Plus, void>(mean, none, red[1]);
    mean /= (float)cols;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int dup = (j * TPR + t) * 8 - (cols - 8);   // columns another chunk owns (8 or more: all)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = KIND == kLayer ? h[j][e] - mean : h[j][e], x = e >= dup ? d : 0.0f;
      if constexpr (KIND != kRows) ss += x * x;
      if constexpr (KIND == kLayer) ds += x;
      if constexpr (row_scaled(SC) && KIND == kRms) top = nan_max(top, fabsf(h[j][e] * w[j][e]));
      if constexpr (row_scaled(SC) && KIND == kRows) top = nan_max(top, fabsf(h[j][e]));
    }
  }
  if constexpr (KIND == kRms) row_reduce<WAVE>(ss, top, row_scaled(SC), red[0]);
  else if constexpr (KIND == kLayer) row_join<WAVE, Plus, Plus>(ss, ds, red[0]);
  else if constexpr (row_scaled(SC)) row_join<WAVE, Most, void>(top, none, red[0]);
  if constexpr (KIND == kRms) rstd = 1.0f / sqrtf(ss / (float)cols + a.eps);
  if constexpr (KIND == kLayer) {
    float shift;
    rstd = 1.0f / sqrtf(centre(ss, ds, (float)cols, shift) + a.eps);
    back = -shift * rstd;
    if (a.mean && t == 0) a.mean[row] = mean + shift;
  }
  // The layer norm stores H now (every wave has its loads behind it) and puts Y in its place.  Weight and bias
  // of two chunks come from the caches: held from the start they left a SIMD 5 waves instead of 8, two
  // workgroups a CU instead of four (16384 x 8192 bf16 with residual to bf16 208 us, late 190, to e4m3 rows
  // 241, late 187; 184 and 174 with over_wave's reductions).  One chunk's wait in registers as they are in memory.
  if constexpr (KIND == kLayer) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int at = (j * TPR + t) * 8, col = min(at, cols - 8);
      if (a.H && at < cols) ep_put8(a.H, DT, row * a.ldh + col, 8, h[j]);
      float lb[8] = {};
      if (a.w_t == TG_F32) {
        ep_get8(a.W, TG_F32, col, 8, w[j]);
        if (a.B) ep_get8(a.B, TG_F32, col, 8, lb);
      } else if constexpr (EARLY) {
        ep_unpack8(DT, rw, w[j]);
        ep_unpack8(DT, rb, lb);
      } else {
        ep_get8(a.W, DT, col, 8, w[j]);
        if (a.B) ep_get8(a.B, DT, col, 8, lb);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) h[j][e] = fmaf(fmaf(h[j][e] - mean, rstd, back), w[j][e], lb[e]);
    }
  }
  float scale = 1.0f, inv = 1.0f;   // S and 1/S
  if constexpr (row_scaled(SC)) {
    float amax = KIND == kRms ? top * rstd : top;
    if (KIND == kLayer || (KIND == kRms && !top_fits(top))) {   // the same for all of the row's threads
      amax = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = nan_max(amax, fabsf(KIND == kRms ? h[j][e] * rstd * w[j][e] : h[j][e]));
      if constexpr (!WAVE && KIND == kRms) __syncthreads();   // every wave has read the first reduction
      if constexpr (KIND == kLayer) row_join<WAVE, Most, void>(amax, none, red[2]);
      else row_reduce<WAVE>(none, amax, true, red[0]);
    }
    scale = row_scale<SC>(amax, a.y_t);
    inv = 1.0f / scale;
    if (t == 0) ((float*)a.S)[row] = scale;
  }
  if (KIND != kRows && a.rstd && t == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int at = (j * TPR + t) * 8, col = min(at, cols - 8);
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = KIND == kRms ? h[j][e] * rstd * w[j][e] : h[j][e];
    if constexpr (SC == TG_SCALE_BLOCK) {   // cols % 32 == 0: a block is 4 adjacent lanes' chunks
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = nan_max(m, fabsf(y[e]));
      m = nan_max(m, __shfl_xor(m, 1));
      m = nan_max(m, __shfl_xor(m, 2));
      m = nan_max(m, kAmaxFloor);
      const bool fine = m < __builtin_inff();
      const int x = block_exp(m, a.y_t);
      inv = fine ? __builtin_ldexpf(1.0f, -x) : __builtin_nanf("");
      if (at < cols && (t & 3) == 0) a.S[row * (a.cols / 32) + at / 32] = fine ? (uint8_t)(x + 127) : 255;
    }
    if (at >= cols) continue;
    if (KIND == kRms && a.H) ep_put8(a.H, DT, row * a.ldh + col, 8, h[j]);
    if constexpr (SC == TG_SCALE_NONE) {
      ep_put8(a.Y, DT, row * a.ldy + col, 8, y);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = row_scaled(SC) ? quotient<KIND>(y[e], scale, inv) : y[e] * inv;
      put_q8(a.Y + row * a.ldy + col, 8, quant8<SC>(y, a.y_t));
    }
  }
}

// Rows outside 8 .. kNormRegCols columns: one workgroup per row, which reads the row twice (the
// second time from the caches).
template <int KIND, int DT, int SC>
__global__ __launch_bounds__(1024) void norm_long(NormArgs a) {
  __shared__ float red[KIND == kLayer ? 3 : 1][16][2];
  const int64_t row = blockIdx.x;
  float mean = 0.0f, back = 0.0f, rstd = 1.0f;
  auto get = [&](int64_t col, int n, float (&h)[8]) {
    ep_get8(a.X, DT, row * a.ldx + col, n, h);
    if (KIND != kRows && a.R) {
      float r[8];
      ep_get8(a.R, DT, row * a.ldr + col, n, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = h[e] + r[e];
        if constexpr (DT == TG_BF16) h[e] = (float)(__bf16)x;
        else if constexpr (DT == TG_F16) h[e] = (float)(_Float16)x;
        else h[e] = x;
      }
    }
  };
  auto weight = [&](int64_t col, int n, float (&w)[8]) {
    if (a.w_t == TG_F32) ep_get8(a.W, TG_F32, col, n, w);
    else ep_get8(a.W, DT, col, n, w);
  };
  float ss = 0.0f, ds = 0.0f, top = 0.0f, none = 0.0f, h[8];
  // Y of a chunk whose H is in h; elements past the row are 0
  auto values = [&](int64_t col, int n, float (&y)[8]) {
    float w[8], b[8] = {};
    if constexpr (KIND != kRows) weight(col, n, w);
    if constexpr (KIND == kLayer) {
      if (a.B && a.w_t == TG_F32) ep_get8(a.B, TG_F32, col, n, b);
      else if (a.B) ep_get8(a.B, DT, col, n, b);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if constexpr (KIND == kRms) y[e] = h[e] * rstd * w[e];
      else if constexpr (KIND == kLayer) y[e] = fmaf(fmaf(h[e] - mean, rstd, back), w[e], b[e]);
      else y[e] = h[e];
  };
  if constexpr (KIND == kLayer) {
    for (int64_t col = (int64_t)threadIdx.x * 8; col < a.cols; col += 8192) {
      get(col, (int)min((int64_t)8, a.cols - col), h);
#pragma unroll
      for (int e = 0; e < 8; ++e) mean += h[e];
    }
    row_join<false, Plus, void>(mean, none, red[1]);
    mean /= (float)a.cols;
  }
  if constexpr (KIND != kRows || row_scaled(SC)) {
    for (int64_t col = (int64_t)threadIdx.x * 8; col < a.cols; col += 8192) {
      const int n = (int)min((int64_t)8, a.cols - col);
      float w[8];
      get(col, n, h);
      if constexpr (row_scaled(SC) && KIND == kRms) weight(col, n, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {   // elements past the row are 0
        const float x = KIND == kLayer ? (e < n ? h[e] - mean : 0.0f) : h[e];
        if constexpr (KIND != kRows) ss += x * x;
        if constexpr (KIND == kLayer) ds += x;
        if constexpr (row_scaled(SC) && KIND == kRms) top = nan_max(top, fabsf(h[e] * w[e]));
        if constexpr (row_scaled(SC) && KIND == kRows) top = nan_max(top, fabsf(h[e]));
      }
    }
    if constexpr (KIND == kRms) row_reduce<false>(ss, top, row_scaled(SC), red[0]);
    else if constexpr (KIND == kLayer) row_join<false, Plus, Plus>(ss, ds, red[0]);
    else row_join<false, Most, void>(top, none, red[0]);
  }
  if constexpr (KIND == kRms) rstd = 1.0f / sqrtf(ss / (float)a.cols + a.eps);
  if constexpr (KIND == kLayer) {
    float shift;
    rstd = 1.0f / sqrtf(centre(ss, ds, (float)a.cols, shift) + a.eps);
    back = -shift * rstd;
    if (a.mean && threadIdx.x == 0) a.mean[row] = mean + shift;
  }
  float scale = 1.0f, inv = 1.0f;   // S and 1/S
  if constexpr (row_scaled(SC)) {
    float amax = KIND == kRms ? top * rstd : top;
    if (KIND == kLayer || (KIND == kRms && !top_fits(top))) {
      amax = 0.0f;
      for (int64_t col = (int64_t)threadIdx.x * 8; col < a.cols; col += 8192) {
        const int n = (int)min((int64_t)8, a.cols - col);
        float y[8];
        get(col, n, h);
        values(col, n, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = nan_max(amax, e < n ? fabsf(y[e]) : 0.0f);
      }
      if constexpr (KIND == kLayer) {
        row_join<false, Most, void>(amax, none, red[2]);
      } else {
        __syncthreads();
        row_reduce<false>(none, amax, true, red[0]);
      }
    }
    scale = row_scale<SC>(amax, a.y_t);
    inv = 1.0f / scale;
    if (threadIdx.x == 0) ((float*)a.S)[row] = scale;
  }
  if (KIND != kRows && a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
  // whole waves take the shuffles: the bound is rounded up to a wave's 512 columns
  for (int64_t col = (int64_t)threadIdx.x * 8; col < (a.cols + 511) / 512 * 512; col += 8192) {
    const int n = (int)max((int64_t)0, min((int64_t)8, a.cols - col));
    float y[8] = {};
    if (n > 0) {
      get(col, n, h);
      values(col, n, y);
    }
    if constexpr (SC == TG_SCALE_BLOCK) {
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = nan_max(m, fabsf(y[e]));
      m = nan_max(m, __shfl_xor(m, 1));
      m = nan_max(m, __shfl_xor(m, 2));
      m = nan_max(m, kAmaxFloor);
      const bool fine = m < __builtin_inff();
      const int x = block_exp(m, a.y_t);
      inv = fine ? __builtin_ldexpf(1.0f, -x) : __builtin_nanf("");
      if (n > 0 && (threadIdx.x & 3) == 0)
        a.S[row * (a.cols / 32) + col / 32] = fine ? (uint8_t)(x + 127) : 255;
    }
    if (n == 0) continue;
    if (KIND != kRows && a.H) ep_put8(a.H, DT, row * a.ldh + col, n, h);
    if constexpr (SC == TG_SCALE_NONE) {
      ep_put8(a.Y, DT, row * a.ldy + col, n, y);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = row_scaled(SC) ? quotient<KIND>(y[e], scale, inv) : y[e] * inv;
      put_q8(a.Y + row * a.ldy + col, n, quant8<SC>(y, a.y_t));
    }
  }
}

// ---- backward --------------------------------------------------------------------------------
// A workgroup walks rows blockIdx.x, + gridDim.x, … (four at a time with one wave per row) and
// keeps its share of dw (and db) in registers; the shares are written once per workgroup and summed by
// sum_rows, so the order is fixed.  The next row sets out before this one is reduced: rows as they
// are held in memory wait in registers (packed for 16-bit types).
template <int DT>
struct Raw8 {
  ep_u32x4 v[DT == TG_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const uint8_t* p, int64_t i) {
    v[0] = load16(p + (DT == TG_F32 ? 4 : 2) * i);
    if constexpr (DT == TG_F32) v[1] = load16(p + 4 * i + 16);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (DT == TG_F32) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = __builtin_bit_cast(float, (uint32_t)v[e / 4][e % 4]);
    } else {
      ep_unpack8(DT, v[0], f);
    }
  }
};
template <int KIND, int DT, int NV, bool WAVE, int MAXT>
__global__ __launch_bounds__(MAXT) void norm_bwd(NormBwdArgs a) {
  constexpr bool LAYER = KIND == kLayer;
  constexpr int RPB = WAVE ? 4 : 1;
  // 1024 threads leave 128 registers: two fp32 rows, or two rows and both sums, do not fit.  Nor does all of one row of
  // the layer norm beside its weights and both sums: 22 registers are spilled there (fp32 29; RMS norm in 16 bits, two
  // rows, 11).  Rows of 8193 to 16384 columns alone: 4096 x 16384 bf16 120 us (3.4 TB/s), 8192 x 8192 97 (4.2).
  constexpr bool AHEAD = !((DT == TG_F32 || LAYER) && MAXT == 1024);
  __shared__ float red[2][WAVE ? 1 : kMaxWaves][2];
  const int TPR = WAVE ? 64 : (int)blockDim.x;
  const int t = WAVE ? (int)threadIdx.x & 63 : (int)threadIdx.x;
  const int cols = (int)a.cols;
  float w[NV][8], dw[NV][8], db[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = min((j * TPR + t) * 8, cols - 8);
    if (a.w_t == TG_F32) ep_get8(a.W, TG_F32, col, 8, w[j]);
    else ep_get8(a.W, DT, col, 8, w[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[j][e] = db[j][e] = 0.0f;
  }
  struct Row {
    Raw8<DT> dy[NV], h[NV], dh[NV];
    float rstd, mean;
  };
  auto load = [&](int64_t row, Row& x) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = min((j * TPR + t) * 8, cols - 8);
      x.dy[j].load(a.dY, row * a.ldy + col);
      x.h[j].load(a.H, row * a.ldh + col);
      if (a.dH) x.dh[j].load(a.dH, row * a.ldd + col);
    }
    x.rstd = a.rstd[row];
    x.mean = LAYER ? a.mean[row] : 0.0f;
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + (WAVE ? threadIdx.x >> 6 : 0);
  Row x;
  if (AHEAD && row < a.rows) load(row, x);
  for (int par = 0; row < a.rows; row += step, par ^= 1) {
    Row next;
    if constexpr (AHEAD) {
      if (row + step < a.rows) load(row + step, next);
    } else {
      load(row, x);
    }
    const float rstd = x.rstd, mean = x.mean;
    auto hat = [&](float v) { return LAYER ? (v - mean) * rstd : v * rstd; };
    float dot = 0.0f, gsum = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int dup = (j * TPR + t) * 8 - (cols - 8);
      float dy[8], h[8];
      x.dy[j].get(dy);
      x.h[j].get(h);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float p = dy[e] * hat(h[e]);   // dY·xh
        dw[j][e] += p;
        dot += e >= dup ? p * w[j][e] : 0.0f;
        if constexpr (LAYER) {
          db[j][e] += dy[e];
          gsum += e >= dup ? dy[e] * w[j][e] : 0.0f;
        }
      }
    }
    if constexpr (LAYER) row_join<WAVE, Plus, Plus>(dot, gsum, red[par]);
    else row_reduce<WAVE>(dot, gsum, false, red[par]);
    const float c = dot / (float)cols, gmean = gsum / (float)cols;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int at = (j * TPR + t) * 8, col = min(at, cols - 8);
      float dx[8], dy[8], h[8];
      x.dy[j].get(dy);
      x.h[j].get(h);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if constexpr (LAYER) dx[e] = rstd * (dy[e] * w[j][e] - gmean - hat(h[e]) * c);
        else dx[e] = rstd * (dy[e] * w[j][e] - h[e] * rstd * c);
      if (a.dH) {
        float dh[8];
        x.dh[j].get(dh);
#pragma unroll
        for (int e = 0; e < 8; ++e) dx[e] += dh[e];
      }
      // dX may be dH, whose loads no barrier waits for: a moved chunk stores only its own columns
      if (at + 8 <= cols) {
        ep_put8(a.dX, DT, row * a.ldx + col, 8, dx);
      } else if (at < cols) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e >= at - col) ep_put(a.dX, DT, row * a.ldx + col + e, dx[e]);
      }
    }
    if constexpr (AHEAD) x = next;
  }
  // this workgroup's share of a gradient
  auto put_share = [&](float* out, float (&v)[NV][8]) {
    if constexpr (WAVE) {
      // the four waves' shares, joined in LDS
      __shared__ float part[4][NV * 512];
      const int wv = (int)threadIdx.x >> 6;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) part[wv][(j * 8 + e) * 64 + t] = v[j][e];
      __syncthreads();
      if (wv == 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int i = (j * 8 + e) * 64 + t;
            v[j][e] = (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
          }
      }
      __syncthreads();
      if (wv != 0) return;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int at = (j * TPR + t) * 8;
      if (at < cols)   // a moved chunk's duplicated columns hold the same sums as their owner's
        ep_put8((uint8_t*)out, TG_F32, (int64_t)blockIdx.x * a.share_ld + min(at, cols - 8), 8, v[j]);
    }
  };
  if (a.dw) put_share(a.dw, dw);
  if (LAYER && a.db) put_share(a.db, db);
}

// Rows outside the register kernel's range: mean(g·xh) of each row first (kLayer: and mean(g) behind it) ...
template <int KIND, int DT>
__global__ __launch_bounds__(1024) void norm_bwd_dot(NormBwdArgs a) {
  constexpr bool LAYER = KIND == kLayer;
  __shared__ float red[16][2];
  const int64_t row = blockIdx.x;
  const float rstd = a.rstd[row], mean = LAYER ? a.mean[row] : 0.0f;
  float dot = 0.0f, gsum = 0.0f;
  for (int64_t col = (int64_t)threadIdx.x * 8; col < a.cols; col += 8192) {
    const int n = (int)min((int64_t)8, a.cols - col);
    float dy[8], h[8], w[8];
    ep_get8(a.dY, DT, row * a.ldy + col, n, dy);
    ep_get8(a.H, DT, row * a.ldh + col, n, h);
    if (a.w_t == TG_F32) ep_get8(a.W, TG_F32, col, n, w);
    else ep_get8(a.W, DT, col, n, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {   // elements past the row have dy = 0 and a finite h
      if constexpr (LAYER) {
        dot += dy[e] * ((h[e] - mean) * rstd) * w[e];
        gsum += dy[e] * w[e];
      } else {
        dot += dy[e] * (h[e] * rstd) * w[e];
      }
    }
  }
  if constexpr (LAYER) row_join<false, Plus, Plus>(dot, gsum, red);
  else row_reduce<false>(dot, gsum, false, red);
  if (threadIdx.x == 0) {
    if constexpr (LAYER) {
      a.dot[2 * row] = dot / (float)a.cols;
      a.dot[2 * row + 1] = gsum / (float)a.cols;
    } else {
      a.dot[row] = dot / (float)a.cols;
    }
  }
}
// ... then dX and dw by panels of 2048 columns (blockIdx.y, and z past kPanels of them), rows shared over
// blockIdx.x.
constexpr int kPanels = 1 << 15;
template <int KIND, int DT>
__global__ __launch_bounds__(256) void norm_bwd_panel(NormBwdArgs a) {
  constexpr bool LAYER = KIND == kLayer;
  const int64_t col = ((int64_t)blockIdx.z * kPanels + blockIdx.y) * 2048 + threadIdx.x * 8;
  if (col >= a.cols) return;
  const int n = (int)min((int64_t)8, a.cols - col);
  float w[8], dw[8] = {}, db[8] = {};
  if (a.w_t == TG_F32) ep_get8(a.W, TG_F32, col, n, w);
  else ep_get8(a.W, DT, col, n, w);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float rstd = a.rstd[row], c = a.dot[LAYER ? 2 * row : row];
    const float mean = LAYER ? a.mean[row] : 0.0f, gmean = LAYER ? a.dot[2 * row + 1] : 0.0f;
    float dy[8], h[8], dx[8];
    ep_get8(a.dY, DT, row * a.ldy + col, n, dy);
    ep_get8(a.H, DT, row * a.ldh + col, n, h);
    if (a.dH) ep_get8(a.dH, DT, row * a.ldd + col, n, dx);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float xh = LAYER ? (h[e] - mean) * rstd : h[e] * rstd;
      dw[e] += dy[e] * xh;
      if constexpr (LAYER) db[e] += dy[e];
      const float g = LAYER ? dy[e] * w[e] - gmean : dy[e] * w[e];
      dx[e] = rstd * (g - xh * c) + (a.dH ? dx[e] : 0.0f);
    }
    ep_put8(a.dX, DT, row * a.ldx + col, n, dx);
  }
  if (a.dw) ep_put8((uint8_t*)a.dw, TG_F32, (int64_t)blockIdx.x * a.share_ld + col, n, dw);
  if (LAYER && a.db) ep_put8((uint8_t*)a.db, TG_F32, (int64_t)blockIdx.x * a.share_ld + col, n, db);
}

// threads of a workgroup that holds a row, nv chunks each: whole waves
unsigned row_threads(int64_t cols, int nv) { return (unsigned)((cols + 512 * nv - 1) / (512 * nv) * 64); }
// threads of a two-pass kernel's workgroup: rows of fewer than 8 columns are one thread's
dim3 long_threads(int64_t cols) { return dim3(cols < 8 ? 64 : 1024); }

// A launch holds fewer than 2^32 threads: more rows than these are cut into launches (each of a
// millisecond or more).  The same over x and y in one launch cost short calls 0.15 us.
constexpr int64_t kLaunchRows = 1 << 21;
// f(first row, number of rows) until an error
template <class F>
hipError_t over_rows(int64_t rows, F f) {
  for (int64_t r = 0; r < rows; r += kLaunchRows) {
    const hipError_t e = f(r, std::min(rows - r, kLaunchRows));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int KIND, int DT, int SC>
hipError_t go_fwd(const NormArgs& a, hipStream_t s) {
  const dim3 rows((unsigned)a.rows), waves((unsigned)((a.rows + 3) / 4));
  const dim3 one(row_threads(a.cols, 1)), two(row_threads(a.cols, 2));
  if (!norm_in_registers(a.cols)) hipLaunchKernelGGL((norm_long<KIND, DT, SC>), rows, long_threads(a.cols), 0, s, a);
  else if (a.cols <= 512) hipLaunchKernelGGL((norm_rows<KIND, DT, 1, SC, true, 256>), waves, dim3(256), 0, s, a);
  else if (a.cols <= 1024) hipLaunchKernelGGL((norm_rows<KIND, DT, 2, SC, true, 256>), waves, dim3(256), 0, s, a);
  else if (a.cols <= 4096) hipLaunchKernelGGL((norm_rows<KIND, DT, 1, SC, false, 512>), rows, one, 0, s, a);
  else if (a.cols <= 8192) hipLaunchKernelGGL((norm_rows<KIND, DT, 2, SC, false, 512>), rows, two, 0, s, a);
  else hipLaunchKernelGGL((norm_rows<KIND, DT, 2, SC, false, 1024>), rows, two, 0, s, a);
  return hipGetLastError();
}
template <int KIND, int DT>
hipError_t go_fwd(const NormArgs& a, int sc, hipStream_t s) {
  if (sc == TG_SCALE_ROW) return a.y_t == TG_I8 ? go_fwd<KIND, DT, kRowInt>(a, s) : go_fwd<KIND, DT, TG_SCALE_ROW>(a, s);
  if (sc == TG_SCALE_BLOCK) return go_fwd<KIND, DT, TG_SCALE_BLOCK>(a, s);
  if constexpr (KIND != kRows) return go_fwd<KIND, DT, TG_SCALE_NONE>(a, s);
  return hipErrorInvalidValue;
}
template <int KIND, int DT>
hipError_t go_bwd(const NormBwdArgs& a, int64_t groups, hipStream_t s) {
  const dim3 g((unsigned)groups);
  if (!norm_in_registers(a.cols)) {
    const int64_t eb = DT == TG_F32 ? 4 : 2;
    const hipError_t e = over_rows(a.rows, [&](int64_t r, int64_t n) {
      NormBwdArgs b = a;
      b.dY += r * a.ldy * eb;
      b.H += r * a.ldh * eb;
      b.rstd += r;
      if (b.mean) b.mean += r;
      b.dot += KIND == kLayer ? 2 * r : r;
      hipLaunchKernelGGL((norm_bwd_dot<KIND, DT>), dim3((unsigned)n), long_threads(a.cols), 0, s, b);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;   // without the dot products there is nothing to read
    const int64_t panels = (a.cols + 2047) / 2048;
    const dim3 over((unsigned)groups, (unsigned)std::min<int64_t>(panels, kPanels), (unsigned)((panels + kPanels - 1) / kPanels));
    hipLaunchKernelGGL((norm_bwd_panel<KIND, DT>), over, dim3(256), 0, s, a);
  } else if (a.cols <= 512) hipLaunchKernelGGL((norm_bwd<KIND, DT, 1, true, 256>), g, dim3(256), 0, s, a);
  else if (a.cols <= 1024) hipLaunchKernelGGL((norm_bwd<KIND, DT, 2, true, 256>), g, dim3(256), 0, s, a);
  else if (a.cols <= 4096) hipLaunchKernelGGL((norm_bwd<KIND, DT, 1, false, 512>), g, dim3(row_threads(a.cols, 1)), 0, s, a);
  else if (a.cols <= 8192) hipLaunchKernelGGL((norm_bwd<KIND, DT, 2, false, 512>), g, dim3(row_threads(a.cols, 2)), 0, s, a);
  else hipLaunchKernelGGL((norm_bwd<KIND, DT, 2, false, 1024>), g, dim3(row_threads(a.cols, 2)), 0, s, a);
  return hipGetLastError();
}

template <int KIND>
hipError_t launch_norm_kind(const NormArgs& all, int dtype, int scale_kind, hipStream_t s) {
  const int64_t eb = dtype == TG_F32 ? 4 : 2, yb = scale_kind == TG_SCALE_NONE ? eb : 1;
  const int64_t sb = scale_kind == TG_SCALE_ROW ? 4 : scale_kind == TG_SCALE_BLOCK ? all.cols / 32 : 0;
  return over_rows(all.rows, [&](int64_t r, int64_t n) {
    NormArgs a = all;
    a.rows = n;
    a.X += r * a.ldx * eb;
    if (a.R) a.R += r * a.ldr * eb;
    if (a.H) a.H += r * a.ldh * eb;
    a.Y += r * a.ldy * yb;
    if (a.S) a.S += r * sb;
    if (a.rstd) a.rstd += r;
    if (a.mean) a.mean += r;
    if (dtype == TG_F32) return go_fwd<KIND, TG_F32>(a, scale_kind, s);
    if (dtype == TG_F16) return go_fwd<KIND, TG_F16>(a, scale_kind, s);
    return go_fwd<KIND, TG_BF16>(a, scale_kind, s);
  });
}

template <int KIND>
hipError_t launch_norm_bwd_kind(const NormBwdArgs& a, int dtype, int64_t groups, hipStream_t s) {
  if (dtype == TG_F32) return go_bwd<KIND, TG_F32>(a, groups, s);
  if (dtype == TG_F16) return go_bwd<KIND, TG_F16>(a, groups, s);
  return go_bwd<KIND, TG_BF16>(a, groups, s);
}

}  // namespace
}  // namespace tg
