// spec_checks.h -- argument checks on the host that the entry points of the
// decode side share (spec_decode.cu, spec_tree.cu).
#pragma once

#include <cstdint>

#include "../../include/spec_decode.h"
#include "launch_decode.h"

namespace specv {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool want32(const void* p) { return p && aligned(p, 4); }  // a required array of 32-bit values
inline bool may32(const void* p) { return aligned(p, 4); }        // an optional one

inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const auto p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return p < q + static_cast<uintptr_t>(nb) && q < p + static_cast<uintptr_t>(na);
}

// Do T rows of na bytes at a and T of nb bytes at b share bytes?  Of one stride, the rows of
// one may lie between those of the other (columns of a fused projection): then
// the columns decide.
inline bool rows_overlap(const void* a, int64_t a_stride, int64_t na, const void* b, int64_t b_stride, int64_t nb, int64_t T) {
  if (!overlap(a, (T - 1) * a_stride + na, b, (T - 1) * b_stride + nb)) return false;
  if (T == 1 || a_stride != b_stride) return true;
  const auto p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  const auto stride = static_cast<uintptr_t>(a_stride);
  const uintptr_t column = p <= q ? (q - p) % stride : (stride - (p - q) % stride) % stride;  // of b's rows, from a's
  return column < static_cast<uintptr_t>(na) || column + static_cast<uintptr_t>(nb) > stride;
}

inline spec_status_t done(cudaError_t e) { return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA; }

inline spec_status_t check_cache(const spec_cache_t* c, CacheView* out) {
  if (!c || c->layers < 1 || c->pages < 0 || c->page_size < 1 || c->heads < 1 || c->head_dim < 1)
    return SPEC_ERR_INVALID_ARG;
  if (c->dtype != SPEC_DTYPE_F32 && c->dtype != SPEC_DTYPE_BF16) return SPEC_ERR_INVALID_ARG;
  if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return SPEC_ERR_INVALID_ARG;
  const int64_t esz = c->dtype == SPEC_DTYPE_BF16 ? 2 : 4;
  const int64_t row = static_cast<int64_t>(c->heads) * c->head_dim;
  if (row > (1 << 20) || c->page_size > (1 << 16) || c->pages > (1 << 26) || c->layers > (1 << 16))
    return SPEC_ERR_UNSUPPORTED;
  if (row * esz % 16) return SPEC_ERR_UNSUPPORTED;  // tokens are copied in 16-byte pieces
  if (c->layer_stride < 0 || c->page_stride < 0 || c->token_stride < row) return SPEC_ERR_INVALID_ARG;
  if (c->layer_stride * esz % 16 || c->page_stride * esz % 16 || c->token_stride * esz % 16)
    return SPEC_ERR_INVALID_ARG;
  // pages, and layers, lie apart (either may be the outer dimension)
  const int64_t span = (c->page_size - 1) * c->token_stride + row;
  if (c->pages > 1 && c->page_stride < span) return SPEC_ERR_INVALID_ARG;
  if (c->layers > 1 && c->layer_stride < span) return SPEC_ERR_INVALID_ARG;
  out->k = static_cast<char*>(c->k);
  out->v = static_cast<char*>(c->v);
  out->layer_stride = c->layer_stride * esz;
  out->page_stride = c->page_stride * esz;
  out->token_stride = c->token_stride * esz;
  out->layers = c->layers;
  out->pages = c->pages;
  out->page_size = c->page_size;
  out->heads = c->heads;
  out->head_dim = c->head_dim;
  out->bf16 = c->dtype == SPEC_DTYPE_BF16;
  return SPEC_OK;
}

inline spec_status_t check_table(const int32_t* ids, int64_t stride, int max_pages, int page_size, PageTable* out) {
  // rows lie apart, or one row (stride 0) holds for every sequence
  if (max_pages < 0 || stride < 0 || (stride > 0 && stride < max_pages) || (max_pages > 0 && !want32(ids)))
    return SPEC_ERR_INVALID_ARG;
  // positions are 32-bit
  if (static_cast<int64_t>(max_pages) * page_size > (1ll << 30)) return SPEC_ERR_UNSUPPORTED;
  out->ids = ids;
  out->stride = stride;
  out->max_pages = max_pages;
  return SPEC_OK;
}

// A workspace of nothing needs no pointer.
inline bool workspace_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws && have >= need && aligned(ws, 16));
}

}  // namespace specv
