// Layer norm and its backward pass, and the quantisation of rows (norm_kernels.h).
#include "norm_kernels.h"

namespace tg {

hipError_t launch_layernorm(const NormArgs& a, int dtype, int scale_kind, hipStream_t s) {
  return launch_norm_kind<kLayer>(a, dtype, scale_kind, s);
}
hipError_t launch_layernorm_bwd(const NormBwdArgs& a, int dtype, int64_t groups, hipStream_t s) {
  return launch_norm_bwd_kind<kLayer>(a, dtype, groups, s);
}
hipError_t launch_quantize_rows(const NormArgs& a, int dtype, int scale_kind, hipStream_t s) {
  return launch_norm_kind<kRows>(a, dtype, scale_kind, s);
}

}  // namespace tg
