// Gated block kernels, 16-bit operands, A [M,K], B [2N,K] or [K,2N].
#include "ep_launch.h"

namespace tg {

hipError_t launch_gated_block(const EpArgs& g, int trans_b, int a_dtype, int b_dtype, const EpKernel& k, hipStream_t s) {
  if (a_dtype == TG_F16)
    return trans_b ? launch_ep_one<false, false, TG_F16, true>(g, k, s) : launch_ep_one<false, true, TG_F16, true>(g, k, s);
  if (a_dtype == TG_BF16)
    return trans_b ? launch_ep_one<false, false, TG_BF16, true>(g, k, s) : launch_ep_one<false, true, TG_BF16, true>(g, k, s);
  return launch_gated_8(g, a_dtype, b_dtype, k, s);
}

}  // namespace tg
