// The kernels around the product with an epilogue that are not block kernels: the join of a split
// sum, the activation's gradient with the bias gradient, and the sum of partial rows.
#include "ep.h"

namespace tg {
namespace {

// D from `splits` partial sums, added in their order (0 of them: P = 0, the K == 0 product).
// 8 columns per thread; bound by the partial sums' bytes, which the block kernels have just
// written.  Four parts' loads are in flight together: one at a time, 16 parts of one row took
// 7.9 us, nearly all of it waiting.
__global__ __launch_bounds__(256) void ep_join(EpArgs g, int64_t chunks) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= chunks) return;
  const int per_row = (g.N + 7) / 8;
  const int row = (int)(i / per_row), col = (int)(i % per_row) * 8;
  EpCols cols;
  ep_cols(g, col, cols);
  float v[8] = {};
  const float* p = g.part + (int64_t)row * g.part_ld + col;
  const int64_t step = (int64_t)g.M * g.part_ld;
  auto add = [&](float4 a, float4 b) {
    v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
    v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
  };
  int s = 0;
  for (; s + 4 <= g.splits; s += 4, p += 4 * step) {
    float4 a[4], b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] = *(const float4*)(p + k * step);
      b[k] = *(const float4*)(p + k * step + 4);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) add(a[k], b[k]);
  }
  for (; s < g.splits; ++s, p += step) add(*(const float4*)p, *(const float4*)(p + 4));
  ep_finish8(g, row, col, cols, v);
}

// dZ = dY·act'(Z), and the column sums of dZ (before its rounding) over the workgroup's rows.
// 64 columns x rows_per rows per workgroup: 8 lanes of 8 columns (a 128-byte line of each row), 32
// rows at a time, eight such in flight.  One pass over dY and Z, bound by memory.
__global__ __launch_bounds__(256) void act_grad(ActGradArgs a) {
  __shared__ float red[32][64 + 1];
  const int lane = (int)threadIdx.x & 7, rl = (int)threadIdx.x >> 3;
  const int col = (int)blockIdx.x * 64 + lane * 8, n = a.N - col;
  const int r0 = (int)blockIdx.y * a.rows_per, r1 = min(a.M, r0 + a.rows_per);
  float sum[8] = {};
  ep_with_act(a.act, [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    auto finish = [&](int64_t r, float (&dy)[8], const float (&z)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (ACT != TG_ACT_NONE) dy[e] *= ep_act_grad<ACT>(z[e]);
        sum[e] += dy[e];
      }
      if (a.dZ) ep_put8(a.dZ, a.t, r * a.N + col, n, dy);
    };
    if (n >= 8) {
      // dZ may be dY or Z: each element is read by the thread that writes it, before it does
      for (int r = r0 + rl; r < r1; r += 256) {
        ep_u32x4 y[8], z[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (r + 32 * k < r1) {
            y[k] = load16(a.dY + 2 * ((int64_t)(r + 32 * k) * a.ldy + col));
            if constexpr (ACT != TG_ACT_NONE) z[k] = load16(a.Z + 2 * ((int64_t)(r + 32 * k) * a.ldz + col));
          }
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (r + 32 * k < r1) {
            float dy[8], zz[8] = {};
            ep_unpack8(a.t, y[k], dy);
            if constexpr (ACT != TG_ACT_NONE) ep_unpack8(a.t, z[k], zz);
            finish(r + 32 * k, dy, zz);
          }
      }
    } else if (n > 0) {
      for (int r = r0 + rl; r < r1; r += 32) {
        float dy[8], zz[8] = {};
        ep_get8(a.dY, a.t, (int64_t)r * a.ldy + col, n, dy);
        if constexpr (ACT != TG_ACT_NONE) ep_get8(a.Z, a.t, (int64_t)r * a.ldz + col, n, zz);
        finish(r, dy, zz);
      }
    }
  });
  if (!a.sums) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) red[rl][lane * 8 + e] = sum[e];
  __syncthreads();
  // 4 threads a column, 8 rows each, then their sums: always in the same order
  const int c = (int)threadIdx.x >> 2, q = (int)threadIdx.x & 3, gc = (int)blockIdx.x * 64 + c;
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) s += red[8 * q + k][c];
  s += __shfl_xor(s, 1);
  s += __shfl_xor(s, 2);
  if (q == 0 && gc < a.N) a.sums[(int64_t)blockIdx.y * a.N + gc] = s;
}

// out[n] = sum over g of part[g][n]: 32 columns x 32 interleaved row lanes per workgroup, joined in
// LDS, always in the same order.  Many lanes a column: the loads wait on memory, not on each other
// (512 rows of 8192 columns: 16 loads a thread).
__global__ __launch_bounds__(1024) void sum_rows(const float* part, int64_t G, int64_t N, float* out) {
  __shared__ float red[32][33];
  const int c = (int)threadIdx.x & 31, l = (int)threadIdx.x >> 5;
  const int64_t n = (int64_t)blockIdx.x * 32 + c;
  float s = 0.0f;
  if (n < N) {
    const float* p = part + (int64_t)l * N + n;
#pragma unroll 8
    for (int64_t g = l; g < G; g += 32, p += 32 * N) s += *p;
  }
  red[l][c] = s;
  __syncthreads();
  // column l of the workgroup by its 32 lanes c
  s = red[c][l];
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) s += __shfl_xor(s, m);
  const int64_t o = (int64_t)blockIdx.x * 32 + l;
  if (c == 0 && o < N) out[o] = s;
}

}  // namespace

hipError_t launch_ep_join(const EpArgs& g, hipStream_t s) {
  const int64_t chunks = (int64_t)g.M * ((g.N + 7) / 8);
  hipLaunchKernelGGL(ep_join, dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, s, g, chunks);
  return hipGetLastError();
}

hipError_t launch_act_grad(const ActGradArgs& a, int groups, hipStream_t s) {
  hipLaunchKernelGGL(act_grad, dim3((unsigned)((a.N + 63) / 64), (unsigned)groups), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_sum_rows(const float* part, int64_t G, int64_t N, float* out, hipStream_t s) {
  hipLaunchKernelGGL(sum_rows, dim3((unsigned)((N + 31) / 32)), dim3(1024), 0, s, part, G, N, out);
  return hipGetLastError();
}

hipError_t launch_ep_block(const EpArgs& g, int trans_a, int trans_b, int a_dtype, int b_dtype,
                           const EpKernel& k, hipStream_t s) {
  if (a_dtype == TG_FP8_E4M3 || a_dtype == TG_FP8_E5M2) return launch_ep_fp8(g, a_dtype, b_dtype, k, s);
  if (trans_a) return trans_b ? launch_ep_mk(g, a_dtype, k, s) : launch_ep_mm(g, a_dtype, k, s);
  return trans_b ? launch_ep_kk(g, a_dtype, k, s) : launch_ep_km(g, a_dtype, k, s);
}

}  // namespace tg
