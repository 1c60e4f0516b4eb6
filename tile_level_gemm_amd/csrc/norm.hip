// Root-mean-square norm with the residual's addition, and its backward pass.
//
//   H = X + R (rounded to X's type: it is the residual stream the next layer reads, and the
//   norm is taken of what that layer will see)   rstd = 1/sqrt(mean(H²) + eps)   Y = H·rstd·w
//   8-bit Y: row scale s = max|Y|/qmax, or per 32 columns the smallest power of two s with
//   max|Y|/s <= qmax, so nothing saturates; Q = Y/s rounded once.  max|Y| is floored at 2^-100.
//   backward: g = dY·w, xh = H·rstd, dX = rstd·(g − xh·mean(g·xh)) + dH, dw = Σ_rows dY·xh.
//
// All of it is bound by memory: one pass, the row kept in registers between the reduction and
// the result, NV chunks of 8 columns a thread.  Rows up to 1024 columns take one wave each and no
// barrier; longer ones a workgroup of as many waves as their chunks need (1003 x 2057: 5 waves of one
// chunk 5.4 us, 4 waves of two 6.2).  The sum of squares and max|H·w| (a row scale needs it:
// max|Y| = rstd·max|H·w|) travel in one reduction; a row whose max|H·w| is out of fp32's range
// (top_fits) takes a second one for max|Y| itself.
// Measured: 16384 x 8192 bf16 with residual to e4m3 blocks 163 us (5.8 TB/s of 944 MB); backward of
// 8192 x 8192 bf16 with dH 100 us and 4 for the sum of dw's shares (5.2 TB/s of 537 MB); one row of
// 4096 2.9 us, launch and latency.
// Rows whose length is not a multiple of 8 end in a chunk moved back to the row's last 8
// columns: every load is a whole vector, and the columns another chunk owns (`dup` of them) are left
// out of the sums.  Forward both owners store the same values; backward, where dX may be dH, a moved
// chunk stores its own columns only.
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

// 8 values to 8-bit floats; |v| <= qmax up to rounding, clamped there; NaN stays NaN
__device__ __forceinline__ uint2 quant8(const float (&v)[8], int t) {
  const float q = t == TG_FP8_E4M3 ? 448.0f : 57344.0f;
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

// Whether rstd·max|H·w| is max|Y|: the product with the weight has neither overflowed nor lost bits
// below the floor of max|Y| (NaN: no).
__device__ __forceinline__ bool top_fits(float top) { return top >= kAmaxFloor && top < __builtin_inff(); }
// Row scale of max|Y| >= the floor; NaN for a row with a NaN or an infinity.
__device__ __forceinline__ float row_scale(float amax, int t) {
  amax = nan_max(amax, kAmaxFloor);
  return amax < __builtin_inff() ? amax / (t == TG_FP8_E4M3 ? 448.0f : 57344.0f) : __builtin_nanf("");
}
// y/s rounded to nearest for inv = 1/s rounded to nearest: Markstein's correction (IBM J. Res. Dev. 34,
// 1990) of the product.  The codes are then the quotient by the very scale that is stored; the product
// alone lands on the other side of a border once in some million codes.  Two operations an element
// (16384 x 8192 bf16 166 us; 164.7 without), where the quotient itself takes ten (172).
__device__ __forceinline__ float quotient(float y, float s, float inv) {
  const float q = y * inv;
  return fmaf(fmaf(-q, s, y), inv, q);
}

// SC: tg_scale_kind of the result
// WAVE: a wave per row, four rows a workgroup; else a workgroup per row.
template <int DT, int NV, int SC, bool WAVE, int MAXT>
__global__ __launch_bounds__(MAXT) void rmsnorm(NormArgs a) {
  __shared__ float red[WAVE ? 1 : kMaxWaves][2];
  const int TPR = WAVE ? 64 : (int)blockDim.x;
  const int t = WAVE ? (int)threadIdx.x & 63 : (int)threadIdx.x;
  const int64_t row = WAVE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
  if (WAVE && row >= a.rows) return;
  const int cols = (int)a.cols;
  float h[NV][8], w[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) ep_get8(a.X, DT, row * a.ldx + min((j * TPR + t) * 8, cols - 8), 8, h[j]);
  if (a.R) {
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
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = min((j * TPR + t) * 8, cols - 8);
    if (a.w_t == TG_F32) ep_get8(a.W, TG_F32, col, 8, w[j]);
    else ep_get8(a.W, DT, col, 8, w[j]);
  }
  float ss = 0.0f, top = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int dup = (j * TPR + t) * 8 - (cols - 8);   // columns another chunk owns (8 or more: all)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = e >= dup ? h[j][e] : 0.0f;
      ss += x * x;
      if constexpr (SC == TG_SCALE_ROW) top = nan_max(top, fabsf(h[j][e] * w[j][e]));
    }
  }
  row_reduce<WAVE>(ss, top, SC == TG_SCALE_ROW, red);
  const float rstd = 1.0f / sqrtf(ss / (float)cols + a.eps);
  float scale = 1.0f, inv = 1.0f;   // S and 1/S
  if constexpr (SC == TG_SCALE_ROW) {
    float amax = top * rstd;
    if (!top_fits(top)) {   // the same for all of the row's threads
      float none = 0.0f;
      amax = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = nan_max(amax, fabsf(h[j][e] * rstd * w[j][e]));
      if constexpr (!WAVE) __syncthreads();   // every wave has read the first reduction
      row_reduce<WAVE>(none, amax, true, red);
    }
    scale = row_scale(amax, a.y_t);
    inv = 1.0f / scale;
    if (t == 0) ((float*)a.S)[row] = scale;
  }
  if (a.rstd && t == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int at = (j * TPR + t) * 8, col = min(at, cols - 8);
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = h[j][e] * rstd * w[j][e];
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
    if (a.H) ep_put8(a.H, DT, row * a.ldh + col, 8, h[j]);
    if constexpr (SC == TG_SCALE_NONE) {
      ep_put8(a.Y, DT, row * a.ldy + col, 8, y);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = SC == TG_SCALE_ROW ? quotient(y[e], scale, inv) : y[e] * inv;
      put_q8(a.Y + row * a.ldy + col, 8, quant8(y, a.y_t));
    }
  }
}

// Rows outside 8 .. kNormRegCols columns: one workgroup per row, which reads the row twice (the
// second time from the caches).
template <int DT, int SC>
__global__ __launch_bounds__(1024) void rmsnorm_long(NormArgs a) {
  __shared__ float red[16][2];
  const int64_t row = blockIdx.x;
  auto get = [&](int64_t col, int n, float (&h)[8], float (&w)[8]) {
    ep_get8(a.X, DT, row * a.ldx + col, n, h);
    if (a.R) {
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
    if (a.w_t == TG_F32) ep_get8(a.W, TG_F32, col, n, w);
    else ep_get8(a.W, DT, col, n, w);
  };
  float ss = 0.0f, top = 0.0f, h[8], w[8];
  for (int64_t col = (int64_t)threadIdx.x * 8; col < a.cols; col += 8192) {
    get(col, (int)min((int64_t)8, a.cols - col), h, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {   // elements past the row are 0
      ss += h[e] * h[e];
      if constexpr (SC == TG_SCALE_ROW) top = nan_max(top, fabsf(h[e] * w[e]));
    }
  }
  row_reduce<false>(ss, top, SC == TG_SCALE_ROW, red);
  const float rstd = 1.0f / sqrtf(ss / (float)a.cols + a.eps);
  float scale = 1.0f, inv = 1.0f;   // S and 1/S
  if constexpr (SC == TG_SCALE_ROW) {
    float amax = top * rstd;
    if (!top_fits(top)) {
      float none = 0.0f;
      amax = 0.0f;
      for (int64_t col = (int64_t)threadIdx.x * 8; col < a.cols; col += 8192) {
        get(col, (int)min((int64_t)8, a.cols - col), h, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = nan_max(amax, fabsf(h[e] * rstd * w[e]));
      }
      __syncthreads();
      row_reduce<false>(none, amax, true, red);
    }
    scale = row_scale(amax, a.y_t);
    inv = 1.0f / scale;
    if (threadIdx.x == 0) ((float*)a.S)[row] = scale;
  }
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
  // whole waves take the shuffles: the bound is rounded up to a wave's 512 columns
  for (int64_t col = (int64_t)threadIdx.x * 8; col < (a.cols + 511) / 512 * 512; col += 8192) {
    const int n = (int)max((int64_t)0, min((int64_t)8, a.cols - col));
    float y[8] = {};
    if (n > 0) {
      get(col, n, h, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = h[e] * rstd * w[e];
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
    if (a.H) ep_put8(a.H, DT, row * a.ldh + col, n, h);
    if constexpr (SC == TG_SCALE_NONE) {
      ep_put8(a.Y, DT, row * a.ldy + col, n, y);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = SC == TG_SCALE_ROW ? quotient(y[e], scale, inv) : y[e] * inv;
      put_q8(a.Y + row * a.ldy + col, n, quant8(y, a.y_t));
    }
  }
}

// ---- backward --------------------------------------------------------------------------------
// A workgroup walks rows blockIdx.x, + gridDim.x, … (four at a time with one wave per row) and
// keeps its share of dw in registers; the shares are written once per workgroup and summed by
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
template <int DT, int NV, bool WAVE, int MAXT>
__global__ __launch_bounds__(MAXT) void rmsnorm_bwd(NormBwdArgs a) {
  constexpr int RPB = WAVE ? 4 : 1;
  // 1024 threads leave 128 registers: two fp32 rows do not fit
  constexpr bool AHEAD = !(DT == TG_F32 && MAXT == 1024);
  __shared__ float red[2][WAVE ? 1 : kMaxWaves][2];
  const int TPR = WAVE ? 64 : (int)blockDim.x;
  const int t = WAVE ? (int)threadIdx.x & 63 : (int)threadIdx.x;
  const int cols = (int)a.cols;
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = min((j * TPR + t) * 8, cols - 8);
    if (a.w_t == TG_F32) ep_get8(a.W, TG_F32, col, 8, w[j]);
    else ep_get8(a.W, DT, col, 8, w[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[j][e] = 0.0f;
  }
  struct Row {
    Raw8<DT> dy[NV], h[NV], dh[NV];
    float rstd;
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
    const float rstd = x.rstd;
    float dot = 0.0f, none = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int dup = (j * TPR + t) * 8 - (cols - 8);
      float dy[8], h[8];
      x.dy[j].get(dy);
      x.h[j].get(h);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float p = dy[e] * (h[e] * rstd);   // dY·xh
        dw[j][e] += p;
        dot += e >= dup ? p * w[j][e] : 0.0f;
      }
    }
    row_reduce<WAVE>(dot, none, false, red[par]);
    const float c = dot / (float)cols;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int at = (j * TPR + t) * 8, col = min(at, cols - 8);
      float dx[8], dy[8], h[8];
      x.dy[j].get(dy);
      x.h[j].get(h);
#pragma unroll
      for (int e = 0; e < 8; ++e) dx[e] = rstd * (dy[e] * w[j][e] - h[e] * rstd * c);
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
  if (!a.dw) return;
  if constexpr (WAVE) {
    // the four waves' shares, joined in LDS
    __shared__ float part[4][NV * 512];
    const int wv = (int)threadIdx.x >> 6;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) part[wv][(j * 8 + e) * 64 + t] = dw[j][e];
    __syncthreads();
    if (wv != 0) return;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = (j * 8 + e) * 64 + t;
        dw[j][e] = (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
      }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int at = (j * TPR + t) * 8;
    if (at < cols)   // a moved chunk's duplicated columns hold the same sums as their owner's
      ep_put8((uint8_t*)a.dw, TG_F32, (int64_t)blockIdx.x * a.cols + min(at, cols - 8), 8, dw[j]);
  }
}

// Rows outside the register kernel's range: mean(g·xh) of each row first ...
template <int DT>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_dot(NormBwdArgs a) {
  __shared__ float red[16][2];
  const int64_t row = blockIdx.x;
  const float rstd = a.rstd[row];
  float dot = 0.0f, none = 0.0f;
  for (int64_t col = (int64_t)threadIdx.x * 8; col < a.cols; col += 8192) {
    const int n = (int)min((int64_t)8, a.cols - col);
    float dy[8], h[8], w[8];
    ep_get8(a.dY, DT, row * a.ldy + col, n, dy);
    ep_get8(a.H, DT, row * a.ldh + col, n, h);
    if (a.w_t == TG_F32) ep_get8(a.W, TG_F32, col, n, w);
    else ep_get8(a.W, DT, col, n, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) dot += dy[e] * (h[e] * rstd) * w[e];
  }
  row_reduce<false>(dot, none, false, red);
  if (threadIdx.x == 0) a.dot[row] = dot / (float)a.cols;
}
// ... then dX and dw by panels of 2048 columns (blockIdx.y, and z past kPanels of them), rows shared over
// blockIdx.x.
constexpr int kPanels = 1 << 15;
template <int DT>
__global__ __launch_bounds__(256) void rmsnorm_bwd_panel(NormBwdArgs a) {
  const int64_t col = ((int64_t)blockIdx.z * kPanels + blockIdx.y) * 2048 + threadIdx.x * 8;
  if (col >= a.cols) return;
  const int n = (int)min((int64_t)8, a.cols - col);
  float w[8], dw[8] = {};
  if (a.w_t == TG_F32) ep_get8(a.W, TG_F32, col, n, w);
  else ep_get8(a.W, DT, col, n, w);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float rstd = a.rstd[row], c = a.dot[row];
    float dy[8], h[8], dx[8];
    ep_get8(a.dY, DT, row * a.ldy + col, n, dy);
    ep_get8(a.H, DT, row * a.ldh + col, n, h);
    if (a.dH) ep_get8(a.dH, DT, row * a.ldd + col, n, dx);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float xh = h[e] * rstd;
      dw[e] += dy[e] * xh;
      dx[e] = rstd * (dy[e] * w[e] - xh * c) + (a.dH ? dx[e] : 0.0f);
    }
    ep_put8(a.dX, DT, row * a.ldx + col, n, dx);
  }
  if (a.dw) ep_put8((uint8_t*)a.dw, TG_F32, (int64_t)blockIdx.x * a.cols + col, n, dw);
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

template <int DT, int SC>
hipError_t go_fwd(const NormArgs& a, hipStream_t s) {
  const dim3 rows((unsigned)a.rows), waves((unsigned)((a.rows + 3) / 4));
  const dim3 one(row_threads(a.cols, 1)), two(row_threads(a.cols, 2));
  if (!norm_in_registers(a.cols)) hipLaunchKernelGGL((rmsnorm_long<DT, SC>), rows, long_threads(a.cols), 0, s, a);
  else if (a.cols <= 512) hipLaunchKernelGGL((rmsnorm<DT, 1, SC, true, 256>), waves, dim3(256), 0, s, a);
  else if (a.cols <= 1024) hipLaunchKernelGGL((rmsnorm<DT, 2, SC, true, 256>), waves, dim3(256), 0, s, a);
  else if (a.cols <= 4096) hipLaunchKernelGGL((rmsnorm<DT, 1, SC, false, 512>), rows, one, 0, s, a);
  else if (a.cols <= 8192) hipLaunchKernelGGL((rmsnorm<DT, 2, SC, false, 512>), rows, two, 0, s, a);
  else hipLaunchKernelGGL((rmsnorm<DT, 2, SC, false, 1024>), rows, two, 0, s, a);
  return hipGetLastError();
}
template <int DT>
hipError_t go_fwd(const NormArgs& a, int sc, hipStream_t s) {
  if (sc == TG_SCALE_ROW) return go_fwd<DT, TG_SCALE_ROW>(a, s);
  if (sc == TG_SCALE_BLOCK) return go_fwd<DT, TG_SCALE_BLOCK>(a, s);
  return go_fwd<DT, TG_SCALE_NONE>(a, s);
}
template <int DT>
hipError_t go_bwd(const NormBwdArgs& a, int64_t groups, hipStream_t s) {
  const dim3 g((unsigned)groups);
  if (!norm_in_registers(a.cols)) {
    const int64_t eb = DT == TG_F32 ? 4 : 2;
    const hipError_t e = over_rows(a.rows, [&](int64_t r, int64_t n) {
      NormBwdArgs b = a;
      b.dY += r * a.ldy * eb;
      b.H += r * a.ldh * eb;
      b.rstd += r;
      b.dot += r;
      hipLaunchKernelGGL((rmsnorm_bwd_dot<DT>), dim3((unsigned)n), long_threads(a.cols), 0, s, b);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;   // without the dot products there is nothing to read
    const int64_t panels = (a.cols + 2047) / 2048;
    const dim3 over((unsigned)groups, (unsigned)std::min<int64_t>(panels, kPanels), (unsigned)((panels + kPanels - 1) / kPanels));
    hipLaunchKernelGGL((rmsnorm_bwd_panel<DT>), over, dim3(256), 0, s, a);
  } else if (a.cols <= 512) hipLaunchKernelGGL((rmsnorm_bwd<DT, 1, true, 256>), g, dim3(256), 0, s, a);
  else if (a.cols <= 1024) hipLaunchKernelGGL((rmsnorm_bwd<DT, 2, true, 256>), g, dim3(256), 0, s, a);
  else if (a.cols <= 4096) hipLaunchKernelGGL((rmsnorm_bwd<DT, 1, false, 512>), g, dim3(row_threads(a.cols, 1)), 0, s, a);
  else if (a.cols <= 8192) hipLaunchKernelGGL((rmsnorm_bwd<DT, 2, false, 512>), g, dim3(row_threads(a.cols, 2)), 0, s, a);
  else hipLaunchKernelGGL((rmsnorm_bwd<DT, 2, false, 1024>), g, dim3(row_threads(a.cols, 2)), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& all, int dtype, int scale_kind, hipStream_t s) {
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
    if (dtype == TG_F32) return go_fwd<TG_F32>(a, scale_kind, s);
    if (dtype == TG_F16) return go_fwd<TG_F16>(a, scale_kind, s);
    return go_fwd<TG_BF16>(a, scale_kind, s);
  });
}

hipError_t launch_rmsnorm_bwd(const NormBwdArgs& a, int dtype, int64_t groups, hipStream_t s) {
  if (dtype == TG_F32) return go_bwd<TG_F32>(a, groups, s);
  if (dtype == TG_F16) return go_bwd<TG_F16>(a, groups, s);
  return go_bwd<TG_BF16>(a, groups, s);
}

}  // namespace tg
