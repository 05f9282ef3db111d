// attention_tree_tc.cu -- the launches of attention_tree_tc.cuh.
#include "attention_tree_tc.cuh"

namespace specv {

size_t tree_tc_workspace(int rows, int D) {
  return static_cast<size_t>(kAttnMaxCtas) * 4 + static_cast<size_t>(ttc::kMaxCtas) * 2 * (rows > 128 ? 256 : 128) * (D + 2) * 4;
}

cudaError_t tree_tc_prepare() {
  cudaError_t e[] = {ttc::prepare<64, false>(), ttc::prepare<64, true>(), ttc::prepare<128, false>(), ttc::prepare<128, true>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

void tree_tc_launch(const AttnArgs& a, int rows, int sm_count, cudaStream_t stream) {
  const bool dual = rows > 128;
  if (a.cache.head_dim == 64) dual ? ttc::launch<64, true>(a, sm_count, stream) : ttc::launch<64, false>(a, sm_count, stream);
  else dual ? ttc::launch<128, true>(a, sm_count, stream) : ttc::launch<128, false>(a, sm_count, stream);
}

}  // namespace specv
