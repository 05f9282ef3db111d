// attention_tc_64.cu -- attention_tc.cuh for heads of 64.
#include "attention_tc.cuh"

namespace specv {

cudaError_t attention_tc_prepare_64() {
  cudaError_t e[] = {tc::prepare<64, 32>(), tc::prepare<64, 48>(), tc::prepare<64, 64>(), tc::prepare<64, 80>(),
                     tc::prepare<64, 96>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

void attention_tc_launch_64(const AttnArgs& a, int n16, int grid, cudaStream_t stream) {
  switch (n16) {
    case 2: tc::launch<64, 32>(a, grid, stream); break;
    case 3: tc::launch<64, 48>(a, grid, stream); break;
    case 4: tc::launch<64, 64>(a, grid, stream); break;
    case 5: tc::launch<64, 80>(a, grid, stream); break;
    default: tc::launch<64, 96>(a, grid, stream); break;
  }
}

}  // namespace specv
