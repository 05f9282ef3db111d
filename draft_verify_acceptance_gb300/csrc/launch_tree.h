// launch_tree.h -- internal host interface between the C ABI of the tree
// operators (spec_tree.cu) and their kernels.
#pragma once

#include "launch_decode.h"

namespace specv {

constexpr int kDataTreeParent = 1024;
constexpr int kDataPathRange = 2048;
constexpr int kMaxNodes = 256;
constexpr int kNodeWords = kMaxNodes / 32;

size_t tree_attention_workspace(int rows, int D, bool bf16);  // rows: of a cache head
cudaError_t tree_attention_prepare();
// tcgen05 kernels (attention_tree_tc.cuh).
size_t tree_tc_workspace(int rows, int D);
cudaError_t tree_tc_prepare();
cudaError_t tree_tc_launch(const AttnArgs& a, int rows, int sm_count, cudaStream_t stream);
cudaError_t launch_tree_attention(const AttnArgs& a, int sm_count, cudaStream_t stream);

struct RotatedAppendArgs {
  const char *k_new, *v_new, *q;
  char* q_out;
  long long new_stride, q_stride, q_out_stride;  // bytes
  int T, B, q_heads, n_freq;
  bool interleaved;
  const int32_t *starts, *positions, *lengths;
  const float* inv_freq;
  CacheView cache;
  PageTable table;
  int32_t* status;
};
cudaError_t launch_rotated_append(const RotatedAppendArgs& a, int sm_count, cudaStream_t stream);

struct AcceptArgs {
  const int32_t *tokens, *parents, *drawn;
  long long parents_stride;
  int B, N;
  int32_t *accepted_len, *out_tokens, *path;
  int32_t* status;
};
cudaError_t launch_tree_accept(const AcceptArgs& a, cudaStream_t stream);

struct KeepArgs {
  CacheView cache;
  PageTable table;
  const int32_t *lengths, *path;
  int B, N;
  int32_t* new_lengths;
  int32_t* status;
};
long long keep_blocks(const CacheView& c);  // a sequence's blocks
cudaError_t launch_keep(const KeepArgs& a, cudaStream_t stream);

}  // namespace specv
