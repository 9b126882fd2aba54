// Tree attention kernels at head_dim 64, the affine codec.
#include "tq_tree_impl.cuh"

namespace tq {

template <>
cudaError_t launch_tree_dim<64, true, false>(const Tables& tb, const CacheView& cv, const TreeArgs& ta, const TreePlan& pl,
                                       uint8_t* ws, cudaLaunchConfig_t* cfg) {
  return dispatch_tree_dim<64, true, false>(tb, cv, ta, pl, ws, cfg);
}

}  // namespace tq
