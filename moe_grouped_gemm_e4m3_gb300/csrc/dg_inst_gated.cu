// dg_inst_gated.cu — instantiations of the gated projection (FP32 scales): BF16/FP32 H. The contiguous
// form; with m_indices null it is the dense one.
#include "dg_launch.h"

namespace dg {
cudaError_t launch_gated(const LaunchArgs& a) {
  return a.out_f32 ? launch_instance<256, kContiguous, true, kSwigluGated>(a)
                   : launch_instance<256, kContiguous, false, kSwigluGated>(a);
}
}  // namespace dg
