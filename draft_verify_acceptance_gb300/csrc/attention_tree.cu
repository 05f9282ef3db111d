// attention_tree.cu -- attention of the nodes of drafted trees over their
// sequences' paged keys and values (sm_103a).
//
//   s_it = scale * q_i . k_t,  out_i = sum_t e^(s_it - m_i) v_t / l_i,
//   l_i = sum_t e^(s_it - m_i),
// over the tokens t before the tree, and those of node i's ancestors and its own.
#include "attention_common.cuh"
#include "attention_mma.cuh"
#include "launch_tree.h"

namespace specv {

// bf16 items of more than 24 rows a cache head (R = N * Hq / Hkv) go to
// attention_tree_tc.cuh, the rest to attention_mma.cuh, in tiles of at most 24 rows
// that each read K and V again (through L2), and scales that are not above zero.
// Measured, mma and tc, 32 query heads on 8, heads of 128:  64 sequences of 400..4000
// tokens, R = 24: 113 and 117 us, R = 32: 181 and 118;  64 of 200..400, R = 32: 55 and 44;
// 8 of 1000, R = 52: 33 and 27;  one of 500, R = 120: 20 and 18, R = 240: 21 and 23;  one
// of 20000, R = 52: 58 and 41.  Heads of 64:  32 of 400..4000, R = 48: 86 and 58;  64 of
// 100..190, two query heads on each, R = 26: 19 and 21.  (tc has since won 2 to 4 us at the small
// ones, 10 at the large.)
namespace {
bool on_tc(int rows, bool bf16) { return bf16 && rows > mma::kMmaRows; }
}  // namespace

size_t tree_attention_workspace(int rows, int D, bool bf16) {
  const size_t bytes = on_tc(rows, bf16) ? tree_tc_workspace(rows, D)
                                         : static_cast<size_t>(kAttnMaxCtas) * 4 + static_cast<size_t>(mma::kMaxMmaCtas) * 2 *
                                                                                       mma::kMmaRows * (D + 2) * 4;
  return (bytes + 255) & ~static_cast<size_t>(255);
}

cudaError_t tree_attention_prepare() {
  cudaError_t e[] = {mma::prepare_all<BF16, 1>(), mma::prepare_all<F32, 1>(), mma::prepare_wide(), tree_tc_prepare()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

cudaError_t launch_tree_attention(const AttnArgs& a, int sm_count, cudaStream_t stream) {
  const int R = a.Q * (a.Hq / a.cache.heads);
  // rows in tiles of equal size
  const int tiles = (R + mma::kMmaRows - 1) / mma::kMmaRows, rows = (R + tiles - 1) / tiles;
  if (on_tc(R, a.cache.bf16) && a.scale_log2 > 0.f) return tree_tc_launch(a, R, sm_count, stream);
  AttnArgs b = a;
  const int nb = (rows + 7) / 8;
  const int64_t items = static_cast<int64_t>(a.B) * a.cache.heads * ((R + 8 * nb - 1) / (8 * nb));
  if (a.cache.bf16) {
    b.whole = a.cache.head_dim == 64 ? mma::whole<BF16, 64, 1>(a, nb, sm_count) : mma::whole<BF16, 128, 1>(a, nb, sm_count);
    mma::launch_rows<BF16, 1>(b, nb, sm_count, stream);
  } else if (a.cache.head_dim == 64 && (mma::whole<F32, 64, 2>(a, nb, sm_count) || items * 4 <= sm_count)) {
    // Few items: an item's tokens by eight warps instead of four.  4 trees of 13 nodes over
    // <= 190 tokens 12.4 -> 10.3 us, 16 over <= 600 21.2 -> 18.3, two of 5 over 3000..5000 24.2 -> 22.8;
    // with more items two blocks of four warps are ahead (8 of 40 nodes over 400..2000 39 us against 45).
    b.whole = mma::whole<F32, 64, 2>(a, nb, sm_count);
    mma::launch_wide(b, nb, sm_count, stream);
  } else {
    b.whole = a.cache.head_dim == 64 ? mma::whole<F32, 64, 1>(a, nb, sm_count) : mma::whole<F32, 128, 1>(a, nb, sm_count);
    mma::launch_rows<F32, 1>(b, nb, sm_count, stream);
  }
  return cudaGetLastError();
}

}  // namespace specv
