// The kernels around the product with an epilogue that are not block kernels: the join of a split
// sum, the activation's gradient with the bias gradient, and the sum of partial rows.
#include "ep.h"

namespace tg {
namespace {

// D from `splits` partial sums, added in their order (0 of them: P = 0, the K == 0 product).
// 8 columns per thread; bound by the partial sums' bytes, which the block kernels have just
// written: two parts of 4096 x 2048, 84 MB, 15.5 us (5.4 TB/s).  Four parts' loads are in flight
// together: one at a time, 16 parts of one row took 7.9 us, nearly all of it waiting.
__global__ __launch_bounds__(256) void ep_join(EpArgs g, int64_t chunks) {
  const int64_t i = wide_block() * 256 + threadIdx.x;
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
// 64 columns x rows_per rows per workgroup: 8 lanes of 8 columns (a 128-byte line of each row), RL
// rows at a time, K such in flight.  One pass over dY and Z, bound by memory: 256 threads with four
// rows each in flight (4096 x 8192: 43 us; 1024 threads with two 51).  A problem that one workgroup per
// 64 columns holds waits for its instructions as well as its rows: there 1024 threads with two
// (200 x 520: 5.4 us; 256 with eight rows 7.3).
// SCALED: a scaled product's gradient, with the scales in registers beside them.
template <int RL, int K, bool SCALED>
__global__ __launch_bounds__(8 * RL) void act_grad(ActGradArgs a) {
  __shared__ float red[RL][64 + 1];
  const int lane = (int)threadIdx.x & 7, rl = (int)threadIdx.x >> 3;
  const int first = ((int)blockIdx.z * kWideRow + (int)blockIdx.x) * 64;   // of the workgroup's columns
  const int col = first + lane * 8, n = a.N - col;
  const int r0 = (int)blockIdx.y * a.rows_per, r1 = min(a.M, r0 + a.rows_per);
  float sum[8] = {}, cs[8];
  if constexpr (SCALED) {
#pragma unroll
    for (int e = 0; e < 8; ++e) cs[e] = 1.0f;
    if (a.cs && n > 0) ep_get8((const uint8_t*)a.cs, TG_F32, col, n, cs);
  }
  // dZ may be dY or Z: each element is read by the thread that writes it, before it does
  ep_with_act(a.act, [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    for (int r = n > 0 ? r0 + rl : r1; r < r1; r += RL * K) {
      ep_u32x4 y[K], z[K];
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (k == 0 || r + RL * k < r1) {
          y[k] = ep_load8_16(a.dY, (int64_t)(r + RL * k) * a.ldy + col, n);
          if constexpr (ACT != TG_ACT_NONE) z[k] = ep_load8_16(a.Z, (int64_t)(r + RL * k) * a.ldz + col, n);
        }
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (k == 0 || r + RL * k < r1) {
          float dy[8], zz[8];
          ep_unpack8(a.t, y[k], dy);
          if constexpr (ACT != TG_ACT_NONE) {
            ep_unpack8(a.t, z[k], zz);
#pragma unroll
            for (int e = 0; e < 8; ++e) dy[e] *= ep_act_grad<ACT>(zz[e]);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] += dy[e];
          if constexpr (SCALED) {
            const float rs = a.rs ? a.rs[r + RL * k] : 1.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) dy[e] = dy[e] * rs * cs[e];
          }
          if (a.dZ) ep_store8_16(a.dZ, (int64_t)(r + RL * k) * a.N + col, n, ep_pack8(a.t, dy));
        }
    }
  });
  if (!a.sums) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) red[rl][lane * 8 + e] = sum[e];
  __syncthreads();
  // RL / 8 threads a column, 8 rows each, then their sums: always in the same order
  constexpr int Q = RL / 8;
  const int c = (int)threadIdx.x / Q, q = (int)threadIdx.x % Q, gc = first + c;
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) s += red[8 * q + k][c];
#pragma unroll
  for (int m = 1; m < Q; m <<= 1) s += __shfl_xor(s, m);
  if (q == 0 && gc < a.N) a.sums[(int64_t)blockIdx.y * a.N + gc] = s;
}

// out[n] = sum over g of part[g][n]: 32 columns x 32 interleaved row lanes per workgroup, joined in
// LDS, always in the same order.  Many lanes a column: the loads wait on memory, not on each other
// (512 rows of 8192 columns: 16 loads a thread).
__global__ __launch_bounds__(1024) void sum_rows(const float* part, int64_t G, int64_t N, float* out) {
  __shared__ float red[32][33];
  const int c = (int)threadIdx.x & 31, l = (int)threadIdx.x >> 5;
  const int64_t first = wide_block() * 32, n = first + c;
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
  const int64_t o = first + l;
  if (c == 0 && o < N) out[o] = s;
}

}  // namespace

hipError_t launch_ep_join(const EpArgs& g, hipStream_t s) {
  const int64_t chunks = (int64_t)g.M * ((g.N + 7) / 8);
  hipLaunchKernelGGL(ep_join, wide_grid((chunks + 255) / 256), dim3(256), 0, s, g, chunks);
  return hipGetLastError();
}

hipError_t launch_act_grad(const ActGradArgs& a, int groups, hipStream_t s) {
  // columns over x and z, rows over y
  const dim3 cols = wide_grid(((int64_t)a.N + 63) / 64), grid(cols.x, (unsigned)groups, cols.y);
  const bool scaled = a.rs || a.cs;
  if (groups == 1) {
    if (scaled) hipLaunchKernelGGL((act_grad<128, 2, true>), grid, dim3(1024), 0, s, a);
    else hipLaunchKernelGGL((act_grad<128, 2, false>), grid, dim3(1024), 0, s, a);
  } else {
    if (scaled) hipLaunchKernelGGL((act_grad<32, 4, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((act_grad<32, 4, false>), grid, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

hipError_t launch_sum_rows(const float* part, int64_t G, int64_t N, float* out, hipStream_t s) {
  hipLaunchKernelGGL(sum_rows, wide_grid((N + 31) / 32), dim3(1024), 0, s, part, G, N, out);
  return hipGetLastError();
}

hipError_t launch_ep_block(const EpArgs& g, int trans_a, int trans_b, int a_dtype, int b_dtype,
                           const EpKernel& k, hipStream_t s) {
  if (a_dtype == TG_FP8_E4M3 || a_dtype == TG_FP8_E5M2) return launch_ep_fp8(g, a_dtype, b_dtype, k, s);
  if (trans_a) return trans_b ? launch_ep_mk(g, a_dtype, k, s) : launch_ep_mm(g, a_dtype, k, s);
  return trans_b ? launch_ep_kk(g, a_dtype, k, s) : launch_ep_km(g, a_dtype, k, s);
}

}  // namespace tg
