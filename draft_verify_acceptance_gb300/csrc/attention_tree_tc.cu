// attention_tree_tc.cu -- the launches of attention_tree_tc.cuh.
#include "attention_tree_tc.cuh"

namespace specv {

size_t tree_tc_workspace(int rows, int D) {
  if (D == 64) return rows > 128 ? ttc::workspace<64, true>() : ttc::workspace<64, false>();
  return rows > 128 ? ttc::workspace<128, true>() : ttc::workspace<128, false>();
}

cudaError_t tree_tc_prepare() {
  cudaError_t e[] = {ttc::prepare<64, false>(), ttc::prepare<64, true>(), ttc::prepare<128, false>(), ttc::prepare<128, true>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

cudaError_t tree_tc_launch(const AttnArgs& a, int rows, int sm_count, cudaStream_t stream) {
  if (a.cache.head_dim == 64)
    return rows > 128 ? ttc::launch<64, true>(a, sm_count, stream) : ttc::launch<64, false>(a, sm_count, stream);
  return rows > 128 ? ttc::launch<128, true>(a, sm_count, stream) : ttc::launch<128, false>(a, sm_count, stream);
}

}  // namespace specv
