// dg_inst_gated.cu — instantiations of the gated projection (FP32 scales): BN 128/256, BF16/FP32 H. The contiguous
// form; with m_indices null it is the dense one.
#include "dg_launch.h"

namespace dg {
cudaError_t launch_gated(const LaunchArgs& a) {
  if (a.block_n == 256)
    return a.out_f32 ? launch_instance<256, kContiguous, true, kSwigluGated>(a)
                     : launch_instance<256, kContiguous, false, kSwigluGated>(a);
  return a.out_f32 ? launch_instance<128, kContiguous, true, kSwigluGated>(a)
                   : launch_instance<128, kContiguous, false, kSwigluGated>(a);
}
}  // namespace dg
