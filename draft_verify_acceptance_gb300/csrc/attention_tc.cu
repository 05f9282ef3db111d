// attention_tc.cu -- the launches of attention_tc.cuh, by rows of an item.
#include "attention_tc.cuh"

namespace specv {

cudaError_t attention_tc_prepare() {
  cudaError_t e[] = {tc::prepare<32>(), tc::prepare<48>(), tc::prepare<64>(), tc::prepare<80>(), tc::prepare<96>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

void attention_tc_launch(const AttnArgs& a, int n16, int grid, cudaStream_t stream) {
  switch (n16) {
    case 2: tc::launch<32>(a, grid, stream); break;
    case 3: tc::launch<48>(a, grid, stream); break;
    case 4: tc::launch<64>(a, grid, stream); break;
    case 5: tc::launch<80>(a, grid, stream); break;
    default: tc::launch<96>(a, grid, stream); break;
  }
}

}  // namespace specv
