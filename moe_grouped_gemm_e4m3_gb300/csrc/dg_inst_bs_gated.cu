// dg_inst_bs_gated.cu — instantiations of the gated projection on the block-scaled kernel (packed
// UE8M0 scales): BF16/FP32 H. The contiguous form; with m_indices null it is the dense one.
#include "dg_launch.h"

namespace dg {
cudaError_t launch_bs_gated(const LaunchArgs& a) {
  return a.out_f32 ? launch_bs_instance<kContiguous, true, kSwigluGated>(a)
                   : launch_bs_instance<kContiguous, false, kSwigluGated>(a);
}
}  // namespace dg
