// attention.cu -- attention of the newest Q tokens of each sequence over its
// paged keys and values (sm_103a).
//
//   s_rt = scale * q_r . k_t,  out_r = sum_t e^(s_rt - m_r) v_t / l_r,
//   l_r = sum_t e^(s_rt - m_r),  m_r a running maximum,
// for the tokens t <= n - Q + i that query i of a sequence of n tokens sees.
#include "attention_common.cuh"
#include "attention_mma.cuh"

namespace specv {

// Rows a cache head (R = Q * Hq / Hkv) choose the bf16 kernel: up to 24 go to
// attention_mma.cuh, more to attention_tc.cuh.  At 64 sequences of 400..4000
// tokens, Hq 32, Hkv 8, D 128 (floor 94 to 96 us) the two took
//   R = 4: 109 and 147 us;  16: 126 and 147;  24: 140 and 178;
//   R = 32: 235 and 180;    68: 360 and 302
// (a fourth block of 8 rows leaves mma without registers; its K and V come
// through L2 once more a block of rows), with D 64 and R = 24: 100 and 149.
size_t attention_workspace(int D, bool bf16) {
  const size_t rows = bf16 ? kMaxRowsTc : mma::kMmaRows;
  return (static_cast<size_t>(kAttnMaxCtas) * 4 + mma::kMaxMmaCtas * 2 * rows * (D + 2) * 4 + 255) &
         ~static_cast<size_t>(255);
}

cudaError_t attention_prepare() {
  cudaError_t e[] = {mma::prepare_all<BF16>(), mma::prepare_all<F32>(), attention_tc_prepare_64(),
                     attention_tc_prepare_128()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

cudaError_t launch_attention(const AttnArgs& a, int sm_count, cudaStream_t stream) {
  const int R = a.Q * (a.Hq / a.cache.heads);
  // rows in tiles of equal size
  const bool few = !a.cache.bf16 || R <= mma::kMmaRows;
  const int most = few ? mma::kMmaRows : kMaxRowsTc;
  const int tiles = (R + most - 1) / most, rows = (R + tiles - 1) / tiles;
  if (!a.cache.bf16) {
    mma::launch_rows<F32>(a, (rows + 7) / 8, sm_count, stream);
  } else if (few) {
    mma::launch_rows<BF16>(a, (rows + 7) / 8, sm_count, stream);
  } else {
    const int n16 = (rows + 15) / 16;  // 2 to 6
    const int grid = sm_count < mma::kMaxMmaCtas ? sm_count : mma::kMaxMmaCtas;
    if (a.cache.head_dim == 128) attention_tc_launch_128(a, n16, grid, stream);
    else attention_tc_launch_64(a, n16, grid, stream);
  }
  return cudaGetLastError();
}

}  // namespace specv
