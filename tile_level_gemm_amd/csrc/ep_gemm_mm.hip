// Block kernels of the product with an epilogue, 16-bit operands, stored A [K,M], B [K,N].
#include "ep_launch.h"

namespace tg {

hipError_t launch_ep_mm(const EpArgs& g, int dtype, const EpKernel& k, hipStream_t s) {
  return launch_ep_layout<true, true>(g, dtype, k, s);
}

}  // namespace tg
