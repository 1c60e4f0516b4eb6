// Block kernels of the product with an epilogue, 16-bit operands, stored A [K,M], B [N,K].
#include "ep_launch.h"

namespace tg {

hipError_t launch_ep_mk(const EpArgs& g, int dtype, const EpKernel& k, hipStream_t s) {
  return launch_ep_layout<true, false>(g, dtype, k, s);
}

}  // namespace tg
