// Block kernels of the product with an epilogue, 16-bit operands, stored A [M,K], B [K,N].
#include "ep_gemm.h"

namespace tg {

hipError_t launch_ep_km(const EpArgs& g, int dtype, const EpKernel& k, hipStream_t s) {
  return launch_ep_layout<false, true>(g, dtype, k, s);
}

}  // namespace tg
