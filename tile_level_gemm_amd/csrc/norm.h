// Norms and the quantisation of rows: launch arguments.  Internal header.
#pragma once

#include <hip/hip_runtime.h>

#include "tg_internal.h"

namespace tg {

// What the kernels of norm_kernels.h compute.
enum NormKind { kRms, kLayer, kRows };

struct NormArgs {
  const uint8_t* X;
  const uint8_t* R;     // residual or NULL
  const uint8_t* W;
  const uint8_t* B;     // layer norm: bias of the weight's type, or NULL
  uint8_t* H;           // X + R, or NULL
  uint8_t* Y;
  uint8_t* S;           // scales: fp32 [rows] or E8M0 [rows][cols/32]
  float* rstd;          // or NULL
  float* mean;          // layer norm: or NULL
  int64_t rows, cols, ldx, ldr, ldh, ldy;
  float eps;
  int32_t w_t, y_t;     // tg_dtype
};
hipError_t launch_rmsnorm(const NormArgs& a, int dtype, int scale_kind, hipStream_t s);
hipError_t launch_layernorm(const NormArgs& a, int dtype, int scale_kind, hipStream_t s);
// X, Y, S; scale_kind row or block
hipError_t launch_quantize_rows(const NormArgs& a, int dtype, int scale_kind, hipStream_t s);

struct NormBwdArgs {
  const uint8_t* dY;
  const uint8_t* H;
  const uint8_t* W;
  const float* rstd;
  const float* mean;    // layer norm
  const uint8_t* dH;    // or NULL
  uint8_t* dX;
  float* dw;            // [groups][cols], share_ld apart; NULL: no weight gradient
  float* db;            // layer norm: as dw, the bias's
  float* dot;           // long rows: mean(g·xh) of each row, [rows]; layer norm: and mean(g), [rows][2]
  int64_t rows, cols, ldy, ldh, ldd, ldx, share_ld;
  int32_t w_t;
};
// Rows of 8 .. kNormRegCols columns stay in registers; others take the two-pass kernels.
constexpr int64_t kNormRegCols = 16384;
inline bool norm_in_registers(int64_t cols) { return cols >= 8 && cols <= kNormRegCols; }
// groups: workgroups that share the rows, each with its own partial dw row
hipError_t launch_rmsnorm_bwd(const NormBwdArgs& a, int dtype, int64_t groups, hipStream_t s);
hipError_t launch_layernorm_bwd(const NormBwdArgs& a, int dtype, int64_t groups, hipStream_t s);

}  // namespace tg
