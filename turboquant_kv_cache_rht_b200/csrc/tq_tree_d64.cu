// Tree attention kernels at head_dim 64, the Lloyd-Max codecs.
#include "tq_tree_impl.cuh"

namespace tq {

template <>
cudaError_t launch_tree_dim<64, false, false>(const Tables& tb, const CacheView& cv, const TreeArgs& ta, const TreePlan& pl,
                                       uint8_t* ws, cudaLaunchConfig_t* cfg) {
  return dispatch_tree_dim<64, false, false>(tb, cv, ta, pl, ws, cfg);
}

}  // namespace tq
