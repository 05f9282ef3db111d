// spec_decode.cu -- the C ABI declared in include/spec_decode.h: argument
// validation on the host and dispatch to the decode-side kernels.
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/spec_decode.h"
#include "launch.h"
#include "launch_decode.h"
#include "spec_checks.h"

namespace {

using namespace specv;

static_assert(specv::kAttnMaxCtas * 4 == SPEC_ATTENTION_ZERO_BYTES, "the arrival counters");
static_assert(specv::kQueueBytes == SPEC_SAMPLE_ZERO_BYTES, "the queue");

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
    if (e == cudaSuccess) e = specv::attention_prepare();
    if (e == cudaSuccess) e = specv::filtered_sample_prepare();
    if (e == cudaSuccess) e = specv::cache_pages_prepare();
    g_err[dev] = e;
  });
  *sms = g_sms[dev];
  return g_err[dev] == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t spec_attention_workspace_size(int B, int Q, int Hq, int heads, int head_dim, int dtype) {
  if (B < 0 || Q < 0 || heads < 1 || Hq < heads || Hq % heads || head_dim < 1) return 0;
  if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16) return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  return specv::attention_workspace(head_dim, dtype == SPEC_DTYPE_BF16);
}

spec_status_t spec_paged_attention(const void* q, int64_t q_batch_stride, int64_t q_token_stride,
                                   int64_t q_head_stride, const spec_cache_t* cache,
                                   const int32_t* page_table, int64_t table_stride, int max_pages,
                                   const int32_t* lengths, int B, int Q, int Hq, float scale,
                                   void* out, float* lse, void* workspace, size_t workspace_bytes,
                                   spec_stream_t stream, int32_t* device_status) {
  SPEC_RANGE("spec_paged_attention");
  specv::AttnArgs a;
  spec_status_t st = check_cache(cache, &a.cache);
  if (st != SPEC_OK) return st;
  st = check_table(page_table, table_stride, max_pages, cache->page_size, &a.table);
  if (st != SPEC_OK) return st;
  if (B < 0 || Q < 0 || Hq < cache->heads || Hq % cache->heads || cache->layers != 1)
    return SPEC_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return SPEC_ERR_INVALID_ARG;
  if (cache->head_dim != 64 && cache->head_dim != 128) return SPEC_ERR_UNSUPPORTED;
  // row indices within a cache head, and output offsets, are 32-bit in the kernels
  if (Q > (1 << 20) || Hq > (1 << 16) || static_cast<int64_t>(Q) * Hq > (1 << 24) || B > (1 << 24))
    return SPEC_ERR_UNSUPPORTED;
  if (B == 0 || Q == 0) return SPEC_OK;
  const int esz = a.cache.bf16 ? 2 : 4;
  if (!q || !aligned(q, 16) || !out || !aligned(out, 16) || !want32(lengths) || !may32(lse) ||
      !may32(device_status))
    return SPEC_ERR_INVALID_ARG;
  if (q_batch_stride < 0 || q_token_stride < 0 || q_head_stride < 0 || q_batch_stride * esz % 16 ||
      q_token_stride * esz % 16 || q_head_stride * esz % 16)
    return SPEC_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, specv::attention_workspace(cache->head_dim, a.cache.bf16)))
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
  a.Q = Q;
  a.Hq = Hq;
  a.scale_log2 = scale * 1.44269504f;
  a.out = out;
  a.lse = lse;
  a.counters = static_cast<unsigned int*>(workspace);
  a.partials = reinterpret_cast<float*>(a.counters + specv::kAttnMaxCtas);
  a.status = device_status;
  return done(specv::launch_attention(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

spec_status_t spec_cache_append(const void* k_new, const void* v_new, int64_t new_stride, int T,
                                const int32_t* starts, const spec_cache_t* cache,
                                const int32_t* page_table, int64_t table_stride, int max_pages,
                                const int32_t* lengths, int B, spec_stream_t stream,
                                int32_t* device_status) {
  SPEC_RANGE("spec_cache_append");
  CacheView c;
  PageTable t;
  spec_status_t st = check_cache(cache, &c);
  if (st != SPEC_OK) return st;
  st = check_table(page_table, table_stride, max_pages, cache->page_size, &t);
  if (st != SPEC_OK) return st;
  if (B < 0 || T < 0 || c.layers != 1) return SPEC_ERR_INVALID_ARG;
  if (T == 0) return SPEC_OK;
  if (B == 0 || (!starts && T % B)) return SPEC_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(c.heads) * c.head_dim;
  const int esz = c.bf16 ? 2 : 4;
  if (!k_new || !v_new || !aligned(k_new, 16) || !aligned(v_new, 16) || new_stride < row ||
      new_stride * esz % 16 || !want32(lengths) || !may32(starts) || !may32(device_status))
    return SPEC_ERR_INVALID_ARG;
  int sms = 0;
  st = device_sms(&sms);
  if (st != SPEC_OK) return st;
  return done(specv::launch_append(static_cast<const char*>(k_new), static_cast<const char*>(v_new),
                                   new_stride * esz, T, starts, c, t, lengths, B, device_status,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

size_t spec_cache_fork_workspace_size(int pages, int C) {
  return pages < 0 || C < 0 ? 0 : specv::fork_workspace(pages, C);
}

spec_status_t spec_cache_fork(const spec_cache_t* cache, const int32_t* page_table,
                              int64_t table_stride, int max_pages, const int32_t* lengths, int B,
                              const int32_t* parents, const int32_t* keep, int C, int room,
                              int32_t* new_table, int32_t* new_lengths, int32_t* ref_counts,
                              int32_t* free_pages, int32_t* n_free, void* workspace,
                              size_t workspace_bytes, spec_stream_t stream, int32_t* device_status) {
  SPEC_RANGE("spec_cache_fork");
  specv::ForkArgs a;
  spec_status_t st = check_cache(cache, &a.cache);
  if (st != SPEC_OK) return st;
  st = check_table(page_table, table_stride, max_pages, cache->page_size, &a.table);
  if (st != SPEC_OK) return st;
  if (B < 0 || C < 0 || room < 0) return SPEC_ERR_INVALID_ARG;
  if (room > (1 << 30) || static_cast<int64_t>(C) * max_pages > (1ll << 31) - 1) return SPEC_ERR_UNSUPPORTED;
  if ((B > 0 && !want32(lengths)) || !may32(device_status) || !want32(n_free)) return SPEC_ERR_INVALID_ARG;
  if (C > 0 && (!want32(parents) || !want32(keep) || !want32(new_lengths) || (max_pages > 0 && !want32(new_table))))
    return SPEC_ERR_INVALID_ARG;
  if (cache->pages > 0 && (!want32(ref_counts) || !want32(free_pages))) return SPEC_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, specv::fork_workspace(cache->pages, C)))
    return SPEC_ERR_INVALID_ARG;
  int sms = 0;
  st = device_sms(&sms);
  if (st != SPEC_OK) return st;
  a.lengths = lengths;
  a.B = B;
  a.parents = parents;
  a.keep = keep;
  a.C = C;
  a.room = room;
  a.new_table = new_table;
  a.new_lengths = new_lengths;
  a.ref_counts = ref_counts;
  a.free_pages = free_pages;
  a.n_free = n_free;
  a.status = device_status;
  return done(specv::launch_fork(a, workspace, sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t spec_cache_compact_workspace_size(int pages) {
  return pages < 0 ? 0 : specv::compact_workspace(pages);
}

spec_status_t spec_cache_compact(const spec_cache_t* cache, const int32_t* page_table,
                                 int64_t table_stride, int max_pages, int B, int32_t* new_table,
                                 int32_t* ref_counts, int32_t* n_live, void* workspace,
                                 size_t workspace_bytes, spec_stream_t stream, int32_t* device_status) {
  SPEC_RANGE("spec_cache_compact");
  specv::CompactArgs a;
  spec_status_t st = check_cache(cache, &a.cache);
  if (st != SPEC_OK) return st;
  st = check_table(page_table, table_stride, max_pages, cache->page_size, &a.table);
  if (st != SPEC_OK) return st;
  if (B < 0) return SPEC_ERR_INVALID_ARG;
  if (static_cast<int64_t>(B) * max_pages > (1ll << 31) - 1) return SPEC_ERR_UNSUPPORTED;
  if (!want32(n_live) || !may32(device_status) || (cache->pages > 0 && !want32(ref_counts)) ||
      (B > 0 && max_pages > 0 && !want32(new_table)))
    return SPEC_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, specv::compact_workspace(cache->pages)))
    return SPEC_ERR_INVALID_ARG;
  int sms = 0;
  st = device_sms(&sms);
  if (st != SPEC_OK) return st;
  a.B = B;
  a.new_table = new_table;
  a.ref_counts = ref_counts;
  a.n_live = n_live;
  a.status = device_status;
  return done(specv::launch_compact(a, workspace, sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t spec_filtered_sample_workspace_size(int R, int V, int dtype) {
  if (R < 0 || V < 1 || V > SPEC_MAX_V || (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16)) return 0;
  return specv::filtered_sample_workspace(R, V, dtype == SPEC_DTYPE_BF16);
}

spec_status_t spec_filtered_sample(const void* logits, int64_t row_stride, const float* uniforms,
                                   int R, int V, int dtype, float temperature, int top_k, float top_p,
                                   float min_p, const float* temperatures, const int32_t* top_ks,
                                   const float* top_ps, const float* min_ps, int32_t* tokens, float* p,
                                   int32_t* n_kept, void* filtered, void* workspace,
                                   size_t workspace_bytes, spec_stream_t stream, int32_t* device_status) {
  SPEC_RANGE("spec_filtered_sample");
  if (R < 0 || V < 1 || (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16)) return SPEC_ERR_INVALID_ARG;
  if (V > SPEC_MAX_V || R > (1 << 24)) return SPEC_ERR_UNSUPPORTED;
  if (!temperatures && !(temperature >= 0.f && std::isfinite(temperature))) return SPEC_ERR_INVALID_ARG;
  if ((!top_ps && std::isnan(top_p)) || (!min_ps && std::isnan(min_p))) return SPEC_ERR_INVALID_ARG;
  if (R == 0) return SPEC_OK;
  const int esz = dtype == SPEC_DTYPE_BF16 ? 2 : 4;
  if (!logits || !aligned(logits, esz) || row_stride < V || !want32(uniforms) || !want32(tokens) ||
      !may32(p) || !may32(n_kept) || !may32(temperatures) || !may32(top_ks) || !may32(top_ps) ||
      !may32(min_ps) || !may32(device_status) || !aligned(filtered, esz))
    return SPEC_ERR_INVALID_ARG;
  // filtered rows may take the logits' place, but a row must not be written over another's logits
  if (filtered && !(filtered == logits && (row_stride == V || R == 1)) &&
      overlap(logits, ((R - 1) * row_stride + V) * esz, filtered, static_cast<int64_t>(R) * V * esz))
    return SPEC_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, specv::filtered_sample_workspace(R, V, esz == 2)))
    return SPEC_ERR_INVALID_ARG;
  int sms = 0;
  const spec_status_t st = device_sms(&sms);  // (sets the kernels' attributes)
  if (st != SPEC_OK) return st;
  specv::SampleArgs a;
  a.logits = logits;
  a.row_stride = row_stride;
  a.uniforms = uniforms;
  a.R = R;
  a.V = V;
  a.bf16 = esz == 2;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.temperatures = temperatures;
  a.top_ks = top_ks;
  a.top_ps = top_ps;
  a.min_ps = min_ps;
  a.tokens = tokens;
  a.p = p;
  a.n_kept = n_kept;
  a.filtered = filtered;
  a.status = device_status;
  return done(specv::launch_filtered_sample(a, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
