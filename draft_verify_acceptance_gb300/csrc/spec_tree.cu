// spec_tree.cu -- the C ABI declared in include/spec_tree.h: argument
// validation on the host and dispatch to the tree operators' kernels.
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/spec_tree.h"
#include "launch.h"
#include "launch_tree.h"
#include "spec_checks.h"

namespace {

using namespace specv;

static_assert(kAttnMaxCtas * 4 == SPEC_TREE_ATTENTION_ZERO_BYTES, "the arrival counters");
static_assert(kMaxNodes == SPEC_TREE_MAX_NODES, "nodes");

constexpr int kMaxDevices = 64;
std::once_flag g_once[kMaxDevices];
int g_sms[kMaxDevices];
cudaError_t g_err[kMaxDevices];

// SM count of the current device; kernel attributes are set on first use.
spec_status_t device_sms(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SPEC_ERR_CUDA;
  std::call_once(g_once[dev], [dev]() {
    cudaError_t e = cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = tree_attention_prepare();
    g_err[dev] = e;
  });
  *sms = g_sms[dev];
  return g_err[dev] == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

// Rows of a tree's parents lie apart, or one row (stride 0) holds for every sequence.
bool parents_ok(const int32_t* parents, int64_t stride, int N) {
  return want32(parents) && (stride == 0 || stride >= N);
}

}  // namespace

extern "C" {

size_t spec_tree_attention_workspace_size(int B, int N, int Hq, int heads, int head_dim, int dtype) {
  if (B < 0 || N < 0 || N > SPEC_TREE_MAX_NODES || heads < 1 || Hq < heads || Hq > (1 << 16) || Hq % heads) return 0;
  if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16) return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  return tree_attention_workspace(N * (Hq / heads), head_dim, dtype == SPEC_DTYPE_BF16);
}

spec_status_t spec_tree_attention(const void* q, int64_t q_batch_stride, int64_t q_token_stride,
                                  int64_t q_head_stride, const spec_cache_t* cache,
                                  const int32_t* page_table, int64_t table_stride, int max_pages,
                                  const int32_t* lengths, const int32_t* parents,
                                  int64_t parents_stride, int B, int N, int Hq, float scale, void* out,
                                  float* lse, void* workspace, size_t workspace_bytes,
                                  spec_stream_t stream, int32_t* device_status) {
  SPEC_RANGE("spec_tree_attention");
  AttnArgs a;
  spec_status_t st = check_cache(cache, &a.cache);
  if (st != SPEC_OK) return st;
  if (B != 0) st = check_table(page_table, table_stride, max_pages, cache->page_size, &a.table);  // (no row needs no table)
  if (st != SPEC_OK) return st;
  if (B < 0 || N < 0 || Hq < cache->heads || Hq % cache->heads || cache->layers != 1) return SPEC_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return SPEC_ERR_INVALID_ARG;
  if (cache->head_dim != 64 && cache->head_dim != 128) return SPEC_ERR_UNSUPPORTED;
  if (N > SPEC_TREE_MAX_NODES || Hq > (1 << 16) || B > (1 << 24)) return SPEC_ERR_UNSUPPORTED;
  if (B == 0 || N == 0) return SPEC_OK;
  const int esz = a.cache.bf16 ? 2 : 4;
  if (!q || !aligned(q, 16) || !out || !aligned(out, 16) || !want32(lengths) || !parents_ok(parents, parents_stride, N) ||
      !may32(lse) || !may32(device_status))
    return SPEC_ERR_INVALID_ARG;
  if (q_batch_stride < 0 || q_token_stride < 0 || q_head_stride < 0 || q_batch_stride * esz % 16 ||
      q_token_stride * esz % 16 || q_head_stride * esz % 16)
    return SPEC_ERR_INVALID_ARG;
  const int64_t D = cache->head_dim;
  if (overlap(q, ((B - 1) * q_batch_stride + (N - 1) * q_token_stride + (Hq - 1) * q_head_stride + D) * esz, out,
              static_cast<int64_t>(B) * N * Hq * D * esz))
    return SPEC_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes,
                    tree_attention_workspace(N * (Hq / cache->heads), cache->head_dim, a.cache.bf16)))
    return SPEC_ERR_INVALID_ARG;
  int sms = 0;
  st = device_sms(&sms);
  if (st != SPEC_OK) return st;
  a.q = static_cast<const char*>(q);
  a.q_batch = q_batch_stride * esz;
  a.q_token = q_token_stride * esz;
  a.q_head = q_head_stride * esz;
  a.lengths = lengths;
  a.B = B;
  a.Q = N;
  a.Hq = Hq;
  a.scale_log2 = scale * 1.44269504f;
  a.out = out;
  a.lse = lse;
  a.counters = static_cast<unsigned int*>(workspace);
  a.partials = reinterpret_cast<float*>(a.counters + kAttnMaxCtas);
  a.status = device_status;
  a.parents = parents;
  a.parents_stride = parents_stride;
  return done(launch_tree_attention(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

spec_status_t spec_cache_append_rotated(const void* k_new, const void* v_new, int64_t new_stride, int T,
                                        const int32_t* starts, const void* q, int64_t q_stride, int q_heads,
                                        void* q_out, int64_t q_out_stride, const int32_t* positions,
                                        const float* inv_freq, int n_freq, int interleaved,
                                        const spec_cache_t* cache, const int32_t* page_table,
                                        int64_t table_stride, int max_pages, const int32_t* lengths, int B,
                                        spec_stream_t stream, int32_t* device_status) {
  SPEC_RANGE("spec_cache_append_rotated");
  RotatedAppendArgs a;
  spec_status_t st = check_cache(cache, &a.cache);
  if (st != SPEC_OK) return st;
  if (B != 0) st = check_table(page_table, table_stride, max_pages, cache->page_size, &a.table);  // (no row needs no table)
  if (st != SPEC_OK) return st;
  if (B < 0 || T < 0 || q_heads < 0 || n_freq < 0 || a.cache.layers != 1) return SPEC_ERR_INVALID_ARG;
  const int D = a.cache.head_dim;
  if (2ll * n_freq > D) return SPEC_ERR_INVALID_ARG;
  if (D % 8 || D > 256 || n_freq % 8 || q_heads > (1 << 16)) return SPEC_ERR_UNSUPPORTED;
  if (T == 0) return SPEC_OK;
  if (B == 0 || (!starts && T % B)) return SPEC_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(a.cache.heads) * D, q_row = static_cast<int64_t>(q_heads) * D;
  const int esz = a.cache.bf16 ? 2 : 4;
  if (!k_new || !v_new || !aligned(k_new, 16) || !aligned(v_new, 16) || new_stride < row || new_stride * esz % 16 ||
      !want32(lengths) || !may32(starts) || !may32(positions) || (n_freq > 0 && !want32(inv_freq)) ||
      !may32(device_status))
    return SPEC_ERR_INVALID_ARG;
  if (q_heads > 0) {
    if (!q || !q_out || !aligned(q, 16) || !aligned(q_out, 16) || q_stride < q_row || q_stride * esz % 16 ||
        q_out_stride < q_row || q_out_stride * esz % 16)
      return SPEC_ERR_INVALID_ARG;
    const int64_t bytes = q_row * esz, span = (T - 1) * q_out_stride * esz + bytes, new_span = ((T - 1) * new_stride + row) * esz;
    if (q == q_out && (q_stride == q_out_stride || T == 1)) {
      // In place: warps read new keys and values while others of the token write its queries.
      if (rows_overlap(q, q_stride * esz, bytes, k_new, new_stride * esz, row * esz, T) ||
          rows_overlap(q, q_stride * esz, bytes, v_new, new_stride * esz, row * esz, T))
        return SPEC_ERR_INVALID_ARG;
    } else if (overlap(q, (T - 1) * q_stride * esz + bytes, q_out, span) || overlap(k_new, new_span, q_out, span) ||
               overlap(v_new, new_span, q_out, span)) {
      return SPEC_ERR_INVALID_ARG;
    }
  }
  int sms = 0;
  st = device_sms(&sms);
  if (st != SPEC_OK) return st;
  a.k_new = static_cast<const char*>(k_new);
  a.v_new = static_cast<const char*>(v_new);
  a.q = static_cast<const char*>(q);
  a.q_out = static_cast<char*>(q_out);
  a.new_stride = new_stride * esz;
  a.q_stride = q_stride * esz;
  a.q_out_stride = q_out_stride * esz;
  a.T = T;
  a.B = B;
  a.q_heads = q_heads;
  a.n_freq = n_freq;
  a.interleaved = interleaved != 0;
  a.starts = starts;
  a.positions = positions;
  a.lengths = lengths;
  a.inv_freq = inv_freq;
  a.status = device_status;
  return done(launch_rotated_append(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

spec_status_t spec_tree_accept(const int32_t* tokens, const int32_t* parents, int64_t parents_stride,
                               const int32_t* drawn, int B, int N, int32_t* accepted_len,
                               int32_t* out_tokens, int32_t* path, spec_stream_t stream,
                               int32_t* device_status) {
  SPEC_RANGE("spec_tree_accept");
  if (B < 0 || N < 0) return SPEC_ERR_INVALID_ARG;
  if (N > SPEC_TREE_MAX_NODES || B > (1 << 24)) return SPEC_ERR_UNSUPPORTED;
  if (B == 0) return SPEC_OK;
  if (!want32(accepted_len) || !may32(device_status)) return SPEC_ERR_INVALID_ARG;
  if (N > 0 && (!want32(tokens) || !parents_ok(parents, parents_stride, N) || !want32(drawn) || !want32(out_tokens) ||
                !want32(path)))
    return SPEC_ERR_INVALID_ARG;
  if (N > 0) {
    // A warp reads its tree whole before it writes: results may take the place of rows that it alone reads.
    const int64_t rows = static_cast<int64_t>(B) * N * 4, shared = ((B - 1) * parents_stride + N) * 4;
    const bool own = parents_stride == N || B == 1;  // no row of parents is another tree's too
    auto clash = [&](const void* in, int64_t bytes, bool same) {
      return overlap(in, bytes, accepted_len, 4ll * B) || (!(same && in == out_tokens) && overlap(in, bytes, out_tokens, rows)) ||
             (!(same && in == path) && overlap(in, bytes, path, rows));
    };
    if (clash(tokens, rows, true) || clash(drawn, rows, true) || clash(parents, shared, own) ||
        overlap(out_tokens, rows, path, rows) || overlap(out_tokens, rows, accepted_len, 4ll * B) ||
        overlap(path, rows, accepted_len, 4ll * B))
      return SPEC_ERR_INVALID_ARG;
  }
  AcceptArgs a;
  a.tokens = tokens;
  a.parents = parents;
  a.drawn = drawn;
  a.parents_stride = parents_stride;
  a.B = B;
  a.N = N;
  a.accepted_len = accepted_len;
  a.out_tokens = out_tokens;
  a.path = path;
  a.status = device_status;
  return done(launch_tree_accept(a, reinterpret_cast<cudaStream_t>(stream)));
}

spec_status_t spec_cache_keep(const spec_cache_t* cache, const int32_t* page_table, int64_t table_stride,
                              int max_pages, const int32_t* lengths, int B, const int32_t* path, int N,
                              int32_t* new_lengths, spec_stream_t stream, int32_t* device_status) {
  SPEC_RANGE("spec_cache_keep");
  KeepArgs a;
  spec_status_t st = check_cache(cache, &a.cache);
  if (st != SPEC_OK) return st;
  if (B != 0) st = check_table(page_table, table_stride, max_pages, cache->page_size, &a.table);  // (no row needs no table)
  if (st != SPEC_OK) return st;
  if (B < 0 || N < 0) return SPEC_ERR_INVALID_ARG;
  if (N > (1 << 20) || B * keep_blocks(a.cache) > (1ll << 31) - 1) return SPEC_ERR_UNSUPPORTED;
  if (B == 0) return SPEC_OK;
  if (!want32(lengths) || !want32(new_lengths) || !may32(device_status) || (N > 0 && !want32(path)) ||
      overlap(lengths, 4ll * B, new_lengths, 4ll * B) || (N > 0 && overlap(path, 4ll * B * N, new_lengths, 4ll * B)) ||
      (max_pages > 0 && overlap(page_table, 4 * ((B - 1) * table_stride + max_pages), new_lengths, 4ll * B)))
    return SPEC_ERR_INVALID_ARG;
  a.lengths = lengths;
  a.path = path;
  a.B = B;
  a.N = N;
  a.new_lengths = new_lengths;
  a.status = device_status;
  return done(launch_keep(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
