// Tree attention kernels at head_dim 128, the affine codec with the sketch.
#include "tq_tree_impl.cuh"

namespace tq {

template <>
cudaError_t launch_tree_dim<128, true, true>(const Tables& tb, const CacheView& cv, const TreeArgs& ta, const TreePlan& pl,
                                       uint8_t* ws, cudaLaunchConfig_t* cfg) {
  return dispatch_tree_dim<128, true, true>(tb, cv, ta, pl, ws, cfg);
}

}  // namespace tq
