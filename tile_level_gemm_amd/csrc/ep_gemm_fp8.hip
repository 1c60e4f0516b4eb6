// Block kernels of the product with an epilogue, fp8 operands, stored A [M,K], B [N,K].
#include "ep_gemm.h"

namespace tg {

hipError_t launch_ep_fp8(const EpArgs& g, int a_dtype, int b_dtype, const EpKernel& k, hipStream_t s) {
  const bool a5 = a_dtype == TG_FP8_E5M2, b5 = b_dtype == TG_FP8_E5M2;
  if (a5 && b5) return launch_ep_one<false, false, fp8_code(1, 1)>(g, k, s);
  if (a5) return launch_ep_one<false, false, fp8_code(1, 0)>(g, k, s);
  if (b5) return launch_ep_one<false, false, fp8_code(0, 1)>(g, k, s);
  return launch_ep_one<false, false, fp8_code(0, 0)>(g, k, s);
}

}  // namespace tg
