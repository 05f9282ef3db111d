// launch_decode.h -- internal host interface between the C ABI of the
// decode-side operators (spec_decode.cu) and their kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace specv {

// Device status bits (the public header's values).
constexpr int kDataPageRange = 64;
constexpr int kDataLengthRange = 128;
constexpr int kDataCacheFull = 256;
constexpr int kDataParamRange = 512;

// One layer set of a paged cache; strides in bytes.
struct CacheView {
  char* k;
  char* v;
  long long layer_stride, page_stride, token_stride;
  int layers, pages, page_size, heads, head_dim;
  bool bf16;
#ifdef __CUDACC__
  __host__ __device__
#endif
  int row_bytes() const { return heads * head_dim * (bf16 ? 2 : 4); }
};

struct PageTable {
  const int32_t* ids;
  long long stride;  // entries between rows
  int max_pages;
};

struct AttnArgs {
  const char* q;
  long long q_batch, q_token, q_head;  // bytes
  CacheView cache;
  PageTable table;
  const int32_t* lengths;
  int B, Q, Hq;
  float scale_log2;  // scale * log2(e)
  void* out;         // [B, Q, Hq, D]
  float* lse;        // [B, Q, Hq] or null
  unsigned int* counters;
  float* partials;
  int32_t* status;
};

struct SampleArgs {
  const void* logits;
  long long row_stride;  // elements
  const float* uniforms;
  int R, V;
  bool bf16;
  float temperature, top_p, min_p;
  int top_k;
  const float* temperatures;
  const int32_t* top_ks;
  const float* top_ps;
  const float* min_ps;
  int32_t* tokens;
  float* p;
  int32_t* n_kept;
  void* filtered;
  int32_t* status;
};

// CTAs an attention launch has at most: its workspace holds one arrival
// counter and two partial results for each.
constexpr int kAttnMaxCtas = 512;
size_t attention_workspace(int D, bool bf16);
cudaError_t attention_prepare();
// tcgen05 attention (attention_tc.cuh): tiles of 16 * n16 rows, at most kMaxRowsTc.
constexpr int kMaxRowsTc = 96;
cudaError_t attention_tc_prepare();
void attention_tc_launch(const AttnArgs& a, int n16, int grid, cudaStream_t stream);
cudaError_t launch_attention(const AttnArgs& a, int sm_count, cudaStream_t stream);

cudaError_t launch_append(const char* k_new, const char* v_new, long long new_stride, int T,
                          const int32_t* starts, const CacheView& c, const PageTable& t,
                          const int32_t* lengths, int B, int32_t* status, cudaStream_t stream);

struct ForkArgs {
  CacheView cache;
  PageTable table;
  const int32_t* lengths;
  int B;
  const int32_t* parents;
  const int32_t* keep;
  int C, room;
  int32_t *new_table, *new_lengths, *ref_counts, *free_pages, *n_free;
  int32_t* status;
};
cudaError_t cache_pages_prepare();
size_t fork_workspace(int pages, int C);
cudaError_t launch_fork(const ForkArgs& a, void* ws, int sm_count, cudaStream_t stream);

struct CompactArgs {
  CacheView cache;
  PageTable table;
  int B;
  int32_t *new_table, *ref_counts, *n_live;
  int32_t* status;
};
size_t compact_workspace(int pages);
cudaError_t launch_compact(const CompactArgs& a, void* ws, int sm_count, cudaStream_t stream);

constexpr int kQueueBytes = 64;  // at the workspace's start: zero between calls
size_t filtered_sample_workspace(int R, int V, bool bf16);
cudaError_t filtered_sample_prepare();
cudaError_t launch_filtered_sample(const SampleArgs& a, void* ws, cudaStream_t stream);

}  // namespace specv
