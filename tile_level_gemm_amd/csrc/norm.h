// Root-mean-square norm: launch arguments.  Internal header.
#pragma once

#include <hip/hip_runtime.h>

#include "tg_internal.h"

namespace tg {

struct NormArgs {
  const uint8_t* X;
  const uint8_t* R;     // residual or NULL
  const uint8_t* W;
  uint8_t* H;           // X + R, or NULL
  uint8_t* Y;
  uint8_t* S;           // scales: fp32 [rows] or E8M0 [rows][cols/32]
  float* rstd;          // or NULL
  int64_t rows, cols, ldx, ldr, ldh, ldy;
  float eps;
  int32_t w_t, y_t;     // tg_dtype
};
hipError_t launch_rmsnorm(const NormArgs& a, int dtype, int scale_kind, hipStream_t s);

struct NormBwdArgs {
  const uint8_t* dY;
  const uint8_t* H;
  const uint8_t* W;
  const float* rstd;
  const uint8_t* dH;    // or NULL
  uint8_t* dX;
  float* dw;            // [groups][cols]; NULL: no weight gradient
  float* dot;           // long rows: mean(g·xh) of each row, [rows]
  int64_t rows, cols, ldy, ldh, ldd, ldx;
  int32_t w_t;
};
// Rows of 8 .. kNormRegCols columns stay in registers; others take the two-pass kernels.
constexpr int64_t kNormRegCols = 16384;
inline bool norm_in_registers(int64_t cols) { return cols >= 8 && cols <= kNormRegCols; }
// groups: workgroups that share the rows, each with its own partial dw row
hipError_t launch_rmsnorm_bwd(const NormBwdArgs& a, int dtype, int64_t groups, hipStream_t s);

}  // namespace tg
