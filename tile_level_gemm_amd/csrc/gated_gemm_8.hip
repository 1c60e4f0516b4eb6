// Gated block kernels, 8-bit operands, A [M,K], B [2N,K].
#include "ep_launch.h"

namespace tg {

hipError_t launch_gated_8(const EpArgs& g, int a_dtype, int b_dtype, const EpKernel& k, hipStream_t s) {
  if (a_dtype == TG_I8) return launch_ep_one<false, false, TG_I8, true>(g, k, s);
  const bool a5 = a_dtype == TG_FP8_E5M2, b5 = b_dtype == TG_FP8_E5M2;
  if (a5 && b5) return launch_ep_one<false, false, fp8_code(1, 1), true>(g, k, s);
  if (a5) return launch_ep_one<false, false, fp8_code(1, 0), true>(g, k, s);
  if (b5) return launch_ep_one<false, false, fp8_code(0, 1), true>(g, k, s);
  return launch_ep_one<false, false, fp8_code(0, 0), true>(g, k, s);
}

}  // namespace tg
