// The 16-row matrix instructions with exchanged operands: Dᵀ = Bᵀ·Aᵀ.  Internal header.
#pragma once

#include "direct_gemm.h"

namespace tg {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;

// b supplies the instruction's first operand: lane l of the result holds row l%16 of A, columns 4(l/16) ..
// 4(l/16)+3 of B.
template <int DT, class F>
__device__ __forceinline__ f32x4 mfma16t(F b, F a, f32x4 c) {
  if constexpr (DT == TG_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), c, 0, 0, 0);
  else if constexpr (DT == TG_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
  else if constexpr (DT == TG_I8)   // integer sums, held as the bits of c's floats
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, b), __builtin_bit_cast(i32x4, a),
                                                                           __builtin_bit_cast(i32x4, c), 0, 0, 0));
  else
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i32x8, b), __builtin_bit_cast(i32x8, a),
                                                            c, DT & 1, (DT & 3) >> 1, 0, 0, 0, 0);
}

}  // namespace
}  // namespace tg
