// Block kernels of the product with an epilogue, 8-bit integer operands, stored A [M,K], B [N,K].
//
// 16 bytes of K a lane as in the 16-bit kernels, so their stages, fragment reads and schedules serve with twice the K:
// v_mfma_i32_32x32x32_i8 in 64- and 128-wide blocks, v_mfma_i32_16x16x64_i8 in the 256-wide ones (ep_fine.h).  The sums
// are exact, and the epilogue turns them to fp32.
#include "ep_launch.h"

namespace tg {

hipError_t launch_ep_i8(const EpArgs& g, const EpKernel& k, hipStream_t s) {
  return launch_ep_one<false, false, TG_I8>(g, k, s);
}

}  // namespace tg
