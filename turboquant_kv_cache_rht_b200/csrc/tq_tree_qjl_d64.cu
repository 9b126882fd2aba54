// Tree attention kernels at head_dim 64, the Lloyd-Max codecs with the sketch.
#include "tq_tree_impl.cuh"

namespace tq {

template <>
cudaError_t launch_tree_dim<64, false, true>(const Tables& tb, const CacheView& cv, const TreeArgs& ta, const TreePlan& pl,
                                       uint8_t* ws, cudaLaunchConfig_t* cfg) {
  return dispatch_tree_dim<64, false, true>(tb, cv, ta, pl, ws, cfg);
}

}  // namespace tq
