// Block kernels of the product with an epilogue, 16-bit operands, stored A [M,K], B [N,K].
#include "ep_gemm.h"

namespace tg {

hipError_t launch_ep_kk(const EpArgs& g, int dtype, const EpKernel& k, hipStream_t s) {
  return launch_ep_layout<false, false>(g, dtype, k, s);
}

}  // namespace tg
