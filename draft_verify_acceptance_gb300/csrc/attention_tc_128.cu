// attention_tc_128.cu -- attention_tc.cuh for heads of 128.
#include "attention_tc.cuh"

namespace specv {

cudaError_t attention_tc_prepare_128() {
  cudaError_t e[] = {tc::prepare<128, 32>(), tc::prepare<128, 48>(), tc::prepare<128, 64>(), tc::prepare<128, 80>(),
                     tc::prepare<128, 96>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

void attention_tc_launch_128(const AttnArgs& a, int n16, int grid, cudaStream_t stream) {
  switch (n16) {
    case 2: tc::launch<128, 32>(a, grid, stream); break;
    case 3: tc::launch<128, 48>(a, grid, stream); break;
    case 4: tc::launch<128, 64>(a, grid, stream); break;
    case 5: tc::launch<128, 80>(a, grid, stream); break;
    default: tc::launch<128, 96>(a, grid, stream); break;
  }
}

}  // namespace specv
