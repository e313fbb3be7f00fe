// dg_inst_gated.cu — instantiations of the gated projection (FP32 scales): dense and contiguous forms,
// BF16/FP32 H.
#include "dg_launch.h"

namespace dg {
cudaError_t launch_gated(const LaunchArgs& a, Mode mode) {
  if (mode == kDense)
    return a.out_f32 ? launch_instance<256, kDense, true, kSwigluGated>(a) : launch_instance<256, kDense, false, kSwigluGated>(a);
  return a.out_f32 ? launch_instance<256, kContiguous, true, kSwigluGated>(a)
                   : launch_instance<256, kContiguous, false, kSwigluGated>(a);
}
}  // namespace dg
