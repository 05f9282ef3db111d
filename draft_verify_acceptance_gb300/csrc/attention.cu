// attention.cu -- attention of the newest Q tokens of each sequence over its
// paged keys and values (sm_103a).
//
//   s_rt = scale * q_r . k_t,  out_r = sum_t e^(s_rt - m_r) v_t / l_r,
//   l_r = sum_t e^(s_rt - m_r),  m_r a running maximum,
// for the tokens t <= n - Q + i that query i of a sequence of n tokens sees.
#include "attention_common.cuh"
#include "attention_mma.cuh"

namespace specv {

// bf16 items of more than 24 rows a cache head (R = Q * Hq / Hkv) over heads of
// 128 go to attention_tc.cuh when the tables have room for kTcTokens tokens a
// sequence and kTcWork tokens times cache heads in all, the rest to
// attention_mma.cuh, in tiles of at most 24 rows that each read K and V again
// (through L2).  Measured, mma and tc:
//   64 sequences of 400..4000 tokens, 8 cache heads, R = 24: 114 and 169 us;
//     R = 32: 185 and 172;  R = 36: 201 and 201;  R = 68: 291 and 257
//   34 of 7406..9512 tokens, 4 cache heads, R = 72: 251 and 197
//   4 of 10000..20000 tokens, 8 cache heads, R = 32: 75 and 71
//   64 of 1000 tokens, 8 cache heads, R = 32: 95 and 101
//   32 of 500..1500 tokens, 8 cache heads, R = 68: 87 and 97
// (an item's start and end cost tc some 10 us, mma 4).  With heads of 64, for
// which a tcgen05 kernel was tried and not kept, mma was ahead at every size:
// 83 sequences of 188..808 tokens, 8 cache heads, R = 48: 67 and 108; 16 of
// 2400 tokens, R = 85: 28 and 58.
constexpr int64_t kTcTokens = 2048, kTcWork = 300000;

size_t attention_workspace(int D, bool bf16) {
  const size_t rows = bf16 ? kMaxRowsTc : mma::kMmaRows;
  return (static_cast<size_t>(kAttnMaxCtas) * 4 + mma::kMaxMmaCtas * 2 * rows * (D + 2) * 4 + 255) &
         ~static_cast<size_t>(255);
}

cudaError_t attention_prepare() {
  cudaError_t e[] = {mma::prepare_all<BF16>(), mma::prepare_all<F32>(), attention_tc_prepare()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

cudaError_t launch_attention(const AttnArgs& a, int sm_count, cudaStream_t stream) {
  const int R = a.Q * (a.Hq / a.cache.heads);
  const int64_t room = static_cast<int64_t>(a.table.max_pages) * a.cache.page_size;
  const bool tc = a.cache.bf16 && a.cache.head_dim == 128 && R > mma::kMmaRows &&
                  room >= kTcTokens && room * a.B * a.cache.heads >= kTcWork;
  // rows in tiles of equal size
  const int most = tc ? kMaxRowsTc : mma::kMmaRows;
  const int tiles = (R + most - 1) / most, rows = (R + tiles - 1) / tiles;
  if (tc)  // tiles of 32 rows at least, a multiple of 16
    attention_tc_launch(a, (rows + 15) / 16, sm_count < mma::kMaxMmaCtas ? sm_count : mma::kMaxMmaCtas, stream);
  else if (a.cache.bf16)
    mma::launch_rows<BF16>(a, (rows + 7) / 8, sm_count, stream);
  else
    mma::launch_rows<F32>(a, (rows + 7) / 8, sm_count, stream);
  return cudaGetLastError();
}

}  // namespace specv
