// Launches of the block kernels of the product with an epilogue.  Internal header; one orientation per
// translation unit.
#pragma once

#include "ep_fine.h"
#include "ep_gemm.h"

namespace tg {
namespace {

// 256-wide blocks: gated products of 16 bits and products of integers on 16-row instructions always, others where
// the caller asks (k.fine: the gradients of a gated product; their operands are never A [K,M] with B [N,K]), so
// that tile_gemm_ep adds in the order it always has.
template <bool A_MN, bool B_MN, int DT, bool GATED = false>
hipError_t launch_ep_one(const EpArgs& g, const EpKernel& k, hipStream_t s) {
  constexpr bool k16 = DT == TG_F16 || DT == TG_BF16, kAlways = (GATED && k16) || DT == TG_I8, kAsked = k16 && !(A_MN && !B_MN);
  const dim3 grid((unsigned)((int64_t)g.tiles_m * g.tiles_n * g.splits)), block(ep_threads(k.bs));
  if (k.staged) {
    if (k.bs == 64) hipLaunchKernelGGL((gemm_ep_staged<A_MN, B_MN, DT, 64, GATED>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((gemm_ep_staged<A_MN, B_MN, DT, 128, GATED>), grid, block, 0, s, g);
  } else if (k.ring) {
    if (k.bs == 64) hipLaunchKernelGGL((gemm_ep_ring<A_MN, B_MN, DT, 64, GATED>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((gemm_ep_ring<A_MN, B_MN, DT, 128, GATED>), grid, block, 0, s, g);
  } else if (k.bs == 128) {
    hipLaunchKernelGGL((gemm_ep_direct<A_MN, B_MN, DT, 128, GATED>), grid, block, 0, s, g);
  } else if constexpr (kAlways) {
    hipLaunchKernelGGL((gemm_ep_fine<A_MN, B_MN, DT, GATED>), grid, block, 0, s, g);
  } else {
    if constexpr (kAsked)
      if (k.fine) {
        hipLaunchKernelGGL((gemm_ep_fine<A_MN, B_MN, DT, false>), grid, block, 0, s, g);
        return hipGetLastError();
      }
    hipLaunchKernelGGL((gemm_ep_direct<A_MN, B_MN, DT, 256, GATED>), grid, block, 0, s, g);
  }
  return hipGetLastError();
}

template <bool A_MN, bool B_MN>
hipError_t launch_ep_layout(const EpArgs& g, int dtype, const EpKernel& k, hipStream_t s) {
  return dtype == TG_F16 ? launch_ep_one<A_MN, B_MN, TG_F16>(g, k, s)
                         : launch_ep_one<A_MN, B_MN, TG_BF16>(g, k, s);
}

}  // namespace
}  // namespace tg
