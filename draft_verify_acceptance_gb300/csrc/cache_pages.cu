// cache_pages.cu -- the paged cache's page handling: append, fork, compact
// (sm_103a).  Copies move 16-byte pieces; page numbers come from counts of
// references recomputed from the tables, so there is no allocator state that
// could drift from them.
#include <climits>

#include "device_common.cuh"
#include "launch_decode.h"

namespace specv {
namespace {

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ void report(int32_t* status, int bits) {
  if (bits && status) atomicOr(status, bits);
}

// ---- append ----------------------------------------------------------------
// One warp per new token: it finds the token's sequence in `starts`, its page
// in the table, and copies the two rows.
__global__ void __launch_bounds__(256)
append_kernel(const char* k_new, const char* v_new, long long new_stride, int T, const int32_t* starts,
              CacheView c, PageTable table, const int32_t* lengths, int B, int32_t* status) {
  const int lane = threadIdx.x & 31;
  const int vecs = c.row_bytes() / 16;
  const int per = starts ? 0 : T / B;
  for (int row = blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5); row < T;
       row += gridDim.x * (blockDim.x / 32)) {
    int b, after;  // sequence, and its new tokens from this one on
    if (starts) {
      int lo = 0, hi = B;  // the last b with starts[b] <= row
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= row) lo = mid;
        else hi = mid;
      }
      b = lo;
      after = starts[b + 1] - row;
      if (starts[b] > row || after <= 0 || starts[b + 1] > T) {  // rows that no sequence claims
        if (lane == 0) report(status, kDataLengthRange);
        continue;
      }
    } else {
      b = row / per;
      after = per - (row - b * per);
    }
    const long long at = static_cast<long long>(lengths[b]) - after;
    if (at < 0 || at >= static_cast<long long>(table.max_pages) * c.page_size) {
      if (lane == 0) report(status, kDataLengthRange);
      continue;
    }
    const int slot = static_cast<int>(at) / c.page_size;
    const int page = table.ids[b * table.stride + slot];
    if (page < 0 || page >= c.pages) {
      if (lane == 0) report(status, kDataPageRange);
      continue;
    }
    const long long off = page * c.page_stride + (static_cast<int>(at) - slot * c.page_size) * c.token_stride;
    const uint4* ks = reinterpret_cast<const uint4*>(k_new + row * new_stride);
    const uint4* vs = reinterpret_cast<const uint4*>(v_new + row * new_stride);
    uint4* kd = reinterpret_cast<uint4*>(c.k + off);
    uint4* vd = reinterpret_cast<uint4*>(c.v + off);
    for (int j = lane; j < vecs; j += 32) {
      kd[j] = __ldg(ks + j);
      vd[j] = __ldg(vs + j);
    }
  }
}

// ---- fork --------------------------------------------------------------------
// Sequence c of the next step, from its parent's row.
struct Child {
  int parent, keep, full, tail, need;  // kept tokens, full pages of them, tokens in the next; pages wanted
  int bad;
};
__device__ __forceinline__ Child child_of(const ForkArgs& a, int c) {
  const int S = a.cache.page_size;
  Child ch;
  ch.bad = 0;
  ch.parent = a.parents[c];
  ch.keep = a.keep[c];
  const bool none = ch.parent == -1 && ch.keep == 0;
  const bool ok = ch.parent >= 0 && ch.parent < a.B && ch.keep >= 0 &&
                  ch.keep <= min(a.lengths[ch.parent], INT_MAX) &&
                  ch.keep <= static_cast<long long>(a.table.max_pages) * S;
  if (!ok) {
    ch.parent = -1;
    ch.keep = 0;
    if (!none) ch.bad = kDataLengthRange;
  }
  ch.full = ch.keep / S;
  ch.tail = ch.keep - ch.full * S;
  const long long need = (static_cast<long long>(ch.keep) + a.room + S - 1) / S;
  if (need > a.table.max_pages) ch.bad |= kDataLengthRange;
  ch.need = static_cast<int>(need < a.table.max_pages ? need : a.table.max_pages);
  return ch;
}
__device__ __forceinline__ int child_page(const ForkArgs& a, const Child& ch, int j) {
  const int p = a.table.ids[ch.parent * a.table.stride + j];
  return p >= 0 && p < a.cache.pages ? p : -1;
}

// Workspace: refs[P], first[P] (cleared before the launch), order[P] the free
// pages ascending, base[C] the first fresh rank of a sequence (sign bit: its
// last page stays), count of free pages.
struct ForkSpace {
  int *refs, *first, *order, *base, *nfree;
};
__host__ __device__ inline ForkSpace fork_space(void* ws, int P, int C) {
  ForkSpace s;
  s.refs = static_cast<int*>(ws);
  s.first = s.refs + P;
  s.order = s.first + P;
  s.base = s.order + P;
  s.nfree = s.base + C;
  return s;
}

// Full references by page, and for partly filled pages the lowest sequence
// ending there, kept as C - c so that 0 means none.
__global__ void __launch_bounds__(256) fork_count_kernel(const ForkArgs a, ForkSpace s) {
  for (int c = blockIdx.x; c < a.C; c += gridDim.x) {
    const Child ch = child_of(a, c);
    int bad = ch.bad;
    for (int j = threadIdx.x; j < ch.full + (ch.tail > 0); j += blockDim.x) {
      const int p = child_page(a, ch, j);
      if (p < 0) bad |= kDataPageRange;
      else if (j < ch.full) atomicAdd(&s.refs[p], 1);
      else atomicMax(&s.first[p], a.C - c);
    }
    report(a.status, bad);
  }
}

// Inclusive scan of one int a thread over the block; `total` its sum.
__device__ __forceinline__ int block_scan(int v, int* scratch, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int x = lane < kPlanThreads / 32 ? scratch[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += o;
    }
    scratch[lane] = x;
  }
  __syncthreads();
  if (warp > 0) incl += scratch[warp - 1];
  *total = scratch[kPlanThreads / 32 - 1];
  return incl;
}

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkArgs a, ForkSpace s) {
  __shared__ int scratch[32];
  const int tid = threadIdx.x, P = a.cache.pages;
  // which last pages stay, and every sequence's first fresh rank
  int fresh_total = 0;
  for (int c0 = 0; c0 < a.C; c0 += kPlanThreads) {
    const int c = c0 + tid;
    int fresh = 0, stays = 0;
    if (c < a.C) {
      const Child ch = child_of(a, c);
      if (ch.tail > 0) {
        const int p = child_page(a, ch, ch.full);
        stays = p >= 0 && s.refs[p] == 0 && s.first[p] == a.C - c;
      }
      fresh = max(0, ch.need - ch.full - stays);
      a.new_lengths[c] = ch.keep;
    }
    int sum;
    const int incl = block_scan(fresh, scratch, &sum);
    if (c < a.C) s.base[c] = (fresh_total + incl - fresh) | (stays ? INT_MIN : 0);
    fresh_total += sum;
  }
  // the free pages ascending; the first of them are given out
  int before = 0;
  for (int p0 = 0; p0 < P; p0 += kPlanThreads) {
    const int p = p0 + tid;
    const int refs = p < P ? s.refs[p] + (s.refs[p] == 0 && s.first[p] > 0) : 1;
    int sum;
    const int incl = block_scan(refs == 0, scratch, &sum);
    if (p < P) {
      const int rank = before + incl - 1;
      if (refs == 0) {
        s.order[rank] = p;
        if (rank >= fresh_total) a.free_pages[rank - fresh_total] = p;
      }
      a.ref_counts[p] = refs + (refs == 0 && rank < fresh_total);
    }
    before += sum;
  }
  const int left = max(0, before - fresh_total);
  for (int i = left + tid; i < P; i += kPlanThreads) a.free_pages[i] = -1;
  if (tid == 0) {
    *a.n_free = left;
    *s.nfree = before;
    if (fresh_total > before) report(a.status, kDataCacheFull);
  }
}

// Writes the rows of the new table and copies the kept tokens of partly
// filled pages that did not stay: block (c, slice), a slice a layer's K or V.
__global__ void __launch_bounds__(256) fork_write_kernel(const ForkArgs a, ForkSpace s) {
  const CacheView& cv = a.cache;
  const int nfree = *s.nfree;
  const int vecs = cv.row_bytes() / 16;
  for (int c = blockIdx.x; c < a.C; c += gridDim.x) {
    const Child ch = child_of(a, c);
    const int packed = s.base[c], base = packed & INT_MAX;
    const int kept = ch.full + (packed < 0);
    if (blockIdx.y == 0) {
      int32_t* row = a.new_table + static_cast<long long>(c) * a.table.max_pages;
      for (int j = threadIdx.x; j < a.table.max_pages; j += blockDim.x) {
        int p = -1;
        if (j < kept) p = child_page(a, ch, j);
        else if (j < ch.need && base + j - kept < nfree) p = s.order[base + j - kept];
        row[j] = p;
      }
    }
    if (ch.tail > 0 && packed >= 0 && ch.full < ch.need && base < nfree) {
      const int from = child_page(a, ch, ch.full), to = s.order[base];
      if (from < 0) continue;
      for (int y = blockIdx.y; y < 2 * cv.layers; y += gridDim.y) {
        char* pool = (y & 1 ? cv.v : cv.k) + (y >> 1) * cv.layer_stride;
        const char* src = pool + from * cv.page_stride;
        char* dst = pool + to * cv.page_stride;
        for (int e = threadIdx.x; e < ch.tail * vecs; e += blockDim.x) {
          const int t = e / vecs;
          const long long at = t * cv.token_stride + (e - t * vecs) * 16;
          *reinterpret_cast<uint4*>(dst + at) = *reinterpret_cast<const uint4*>(src + at);
        }
      }
    }
  }
}

// ---- compact -------------------------------------------------------------------
// Workspace: refs[P] (cleared before the launch), to[P] the pages' new
// numbers, from[P] the moved pages ascending, holes[P], moves.
struct CompactSpace {
  int *refs, *to, *from, *holes, *moves;
};
__host__ __device__ inline CompactSpace compact_space(void* ws, int P) {
  CompactSpace s;
  s.refs = static_cast<int*>(ws);
  s.to = s.refs + P;
  s.from = s.to + P;
  s.holes = s.from + P;
  s.moves = s.holes + P;
  return s;
}

__global__ void __launch_bounds__(256) compact_count_kernel(const CompactArgs a, CompactSpace s) {
  for (int b = blockIdx.x; b < a.B; b += gridDim.x)
    for (int j = threadIdx.x; j < a.table.max_pages; j += blockDim.x) {
      const int p = a.table.ids[b * a.table.stride + j];
      if (p >= a.cache.pages) report(a.status, kDataPageRange);
      else if (p >= 0) atomicAdd(&s.refs[p], 1);
    }
}

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactArgs a, CompactSpace s) {
  __shared__ int scratch[32];
  const int tid = threadIdx.x, P = a.cache.pages;
  int mine = 0, n;
  for (int p = tid; p < P; p += kPlanThreads) mine += s.refs[p] > 0;
  block_scan(mine, scratch, &n);
  int moves = 0, holes = 0;
  for (int p0 = 0; p0 < P; p0 += kPlanThreads) {
    const int p = p0 + tid;
    const bool live = p < P && s.refs[p] > 0;
    const bool mover = live && p >= n, hole = p < n && !live;
    int sum;
    int incl = block_scan(mover, scratch, &sum);
    if (mover) s.from[moves + incl - 1] = p;
    moves += sum;
    incl = block_scan(hole, scratch, &sum);
    if (hole) s.holes[holes + incl - 1] = p;
    holes += sum;
    if (p < P && !mover) {
      s.to[p] = p;
      if (!hole) a.ref_counts[p] = p < n ? s.refs[p] : 0;
    }
    if (mover) a.ref_counts[p] = 0;
  }
  __syncthreads();
  for (int i = tid; i < moves; i += kPlanThreads) {
    const int from = s.from[i], to = s.holes[i];
    s.to[from] = to;
    a.ref_counts[to] = s.refs[from];
  }
  if (tid == 0) {
    *a.n_live = n;
    *s.moves = moves;
  }
}

__global__ void __launch_bounds__(256) compact_move_kernel(const CompactArgs a, CompactSpace s) {
  const CacheView& cv = a.cache;
  const int P = cv.pages;
  for (int b = blockIdx.x; b < a.B; b += gridDim.x)
    for (int j = threadIdx.x; j < a.table.max_pages; j += blockDim.x) {
      const int p = a.table.ids[b * a.table.stride + j];
      a.new_table[static_cast<long long>(b) * a.table.max_pages + j] = p >= 0 && p < P ? s.to[p] : -1;
    }
  const int moves = *s.moves, vecs = cv.row_bytes() / 16;
  const long long jobs = static_cast<long long>(moves) * cv.layers * 2;
  for (long long x = blockIdx.x; x < jobs; x += gridDim.x) {
    const int i = static_cast<int>(x / (cv.layers * 2)), y = static_cast<int>(x - static_cast<long long>(i) * cv.layers * 2);
    char* pool = (y & 1 ? cv.v : cv.k) + (y >> 1) * cv.layer_stride;
    const char* src = pool + s.from[i] * cv.page_stride;
    char* dst = pool + s.holes[i] * cv.page_stride;
    for (int e = threadIdx.x; e < cv.page_size * vecs; e += blockDim.x) {
      const int t = e / vecs;
      const long long at = t * cv.token_stride + (e - t * vecs) * 16;
      *reinterpret_cast<uint4*>(dst + at) = *reinterpret_cast<const uint4*>(src + at);
    }
  }
}

size_t up(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

}  // namespace

cudaError_t launch_append(const char* k_new, const char* v_new, long long new_stride, int T,
                          const int32_t* starts, const CacheView& c, const PageTable& t,
                          const int32_t* lengths, int B, int32_t* status, int sm_count,
                          cudaStream_t stream) {
  const int blocks = (T + 7) / 8, most = sm_count * 8;
  append_kernel<<<blocks < most ? blocks : most, 256, 0, stream>>>(k_new, v_new, new_stride, T, starts, c, t,
                                                                   lengths, B, status);
  return cudaGetLastError();
}

size_t fork_workspace(int pages, int C) {
  return up((3 * static_cast<size_t>(pages) + static_cast<size_t>(C) + 1) * 4);
}

cudaError_t launch_fork(const ForkArgs& a, void* ws, int sm_count, cudaStream_t stream) {
  const ForkSpace s = fork_space(ws, a.cache.pages, a.C);
  cudaError_t e = cudaMemsetAsync(s.refs, 0, 2 * static_cast<size_t>(a.cache.pages) * 4, stream);
  if (e != cudaSuccess) return e;
  const int blocks = a.C < sm_count * 8 ? a.C : sm_count * 8;
  if (blocks > 0) fork_count_kernel<<<blocks, 256, 0, stream>>>(a, s);
  fork_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, s);
  const int slices = 2 * a.cache.layers < 64 ? 2 * a.cache.layers : 64;
  if (blocks > 0) fork_write_kernel<<<dim3(blocks, slices), 256, 0, stream>>>(a, s);
  return cudaGetLastError();
}

size_t compact_workspace(int pages) { return up((4 * static_cast<size_t>(pages) + 1) * 4); }

cudaError_t launch_compact(const CompactArgs& a, void* ws, int sm_count, cudaStream_t stream) {
  const CompactSpace s = compact_space(ws, a.cache.pages);
  cudaError_t e = cudaMemsetAsync(s.refs, 0, static_cast<size_t>(a.cache.pages) * 4, stream);
  if (e != cudaSuccess) return e;
  const int blocks = a.B < sm_count * 8 ? a.B : sm_count * 8;
  if (blocks > 0) compact_count_kernel<<<blocks, 256, 0, stream>>>(a, s);
  compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, s);
  compact_move_kernel<<<sm_count * 8, 256, 0, stream>>>(a, s);
  return cudaGetLastError();
}

}  // namespace specv
