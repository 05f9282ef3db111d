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
// Both measured on one machine (mma, tc in us; 32 query heads on 8, heads of 128 where not said):
//                                           R = 8      16         24         32 and more
//   64 sequences of 400..4000 tokens        102, 106   107, 106   112, 107   32: 181, 110   64: 288, 112
//   64 of 200..400                           29, 39     36, 39     42, 39    32: 55, 39
//   8 of 1000                                17, 22     23, 22     31, 22    52: 33, 23
//   one of 500                               12, 16     16, 16     19, 16    120: 20, 17   240: 21, 25
//   one of 20000                             33, 35     43, 35     46, 35    52: 58, 36
//   32 of 400..4000, heads of 64             44, 53     47, 53     52, 54    48: 86, 55
//   64 of 100..190, 16 heads of 64 on 8      16, 27     19, 28     21, 28    26: 31, 28
// So 24, a row tile of mma's, is right for heads of 64.  For heads of 128 tc is ahead
// from 17 to 20 rows on, by 5 % for large batches and by 10 to 30 % for small ones, which this
// rule does not take; and behind at 240 rows of one short sequence.
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
