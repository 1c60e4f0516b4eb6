// Root-mean-square norm and its backward pass (norm_kernels.h).
#include "norm_kernels.h"

namespace tg {

hipError_t launch_rmsnorm(const NormArgs& a, int dtype, int scale_kind, hipStream_t s) {
  return launch_norm_kind<kRms>(a, dtype, scale_kind, s);
}
hipError_t launch_rmsnorm_bwd(const NormBwdArgs& a, int dtype, int64_t groups, hipStream_t s) {
  return launch_norm_bwd_kind<kRms>(a, dtype, groups, s);
}

}  // namespace tg
