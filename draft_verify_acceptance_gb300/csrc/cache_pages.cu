// cache_pages.cu -- the paged cache's page handling: append, fork, compact
// (sm_103a).  Copies move 16-byte pieces; page numbers come from counts of
// references recomputed from the tables, so there is no allocator state that
// could drift from them.
//
// fork and compact first make a plan (reference counts, free pages, who gets
// which) and then copy.  Where the counts fit one block's shared memory, one
// block plans there, and the kernel that writes the tables and copies is its
// programmatic dependent: two launches instead of four (a cooperative launch
// of both in one costs the host more than the second launch does), and no
// traffic through L2 for the counts.  Larger pools count in global memory.
#include <climits>

#include "device_common.cuh"
#include "launch_decode.h"

namespace specv {
namespace {

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ void report(int32_t* status, int bits) {
  if (bits && status) atomicOr(status, bits);
}

constexpr int kGroup = 128;            // threads that share a copy
constexpr int kMaxShared = 200 * 1024;  // of the plan

// Waits for what the launch before this one wrote (a dependent launch).
__device__ __forceinline__ void after_plan() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Copies `tokens` tokens of a page by kGroup threads, eight pieces a thread
// in flight where the tokens are contiguous.
__device__ __forceinline__ void copy_tokens(const CacheView& cv, const char* src, char* dst, int tokens, int vecs,
                                            int lane) {
  const int total = tokens * vecs;
  if (cv.token_stride == vecs * 16) {
    const uint4* from = reinterpret_cast<const uint4*>(src) + lane;
    uint4* to = reinterpret_cast<uint4*>(dst) + lane;
    int left = total - lane;
    for (; left > 7 * kGroup; left -= 8 * kGroup, from += 8 * kGroup, to += 8 * kGroup) {
      uint4 w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = from[i * kGroup];
#pragma unroll
      for (int i = 0; i < 8; ++i) to[i * kGroup] = w[i];
    }
    for (; left > 0; left -= kGroup, from += kGroup, to += kGroup) *to = *from;
  } else {
    for (int e = lane; e < total; e += kGroup) {
      const int t = e / vecs;
      const long long at = t * cv.token_stride + (e - t * vecs) * 16;
      *reinterpret_cast<uint4*>(dst + at) = *reinterpret_cast<const uint4*>(src + at);
    }
  }
}

// ---- append ----------------------------------------------------------------
// One warp per new token: it finds the token's sequence in `starts`, its page
// in the table, and copies the two rows.  The rows' first pieces are under way
// while it looks (four dependent loads or more): 53000 tokens of twelve
// sequences, 8 heads of 128, in 55 to 68 us by machine, their bytes at the copy
// rate 54, and a verify step's 384 in 5.5, nearly all of it a launch.
constexpr int kPieces = 4;  // of K, and of V, a lane holds
__global__ void __launch_bounds__(256)
append_kernel(const char* k_new, const char* v_new, long long new_stride, int T, const int32_t* starts,
              CacheView c, PageTable table, const int32_t* lengths, int B, int32_t* status) {
  const int lane = threadIdx.x & 31;
  const int vecs = c.row_bytes() / 16;
  const int per = starts ? 0 : T / B;
  const long long warp = static_cast<long long>(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5);
  if (warp >= T) return;
  const int row = static_cast<int>(warp);
  const uint4* ks = reinterpret_cast<const uint4*>(k_new + row * new_stride) + lane;
  const uint4* vs = reinterpret_cast<const uint4*>(v_new + row * new_stride) + lane;
  uint4 kw[kPieces], vw[kPieces];
  auto load = [&](int j0) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (j0 + i * 32 + lane < vecs) {
        kw[i] = ld_stream_v4(ks + j0 + i * 32);
        vw[i] = ld_stream_v4(vs + j0 + i * 32);
      }
  };
  load(0);
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
      return;
    }
  } else {
    b = row / per;
    after = per - (row - b * per);
  }
  const long long at = static_cast<long long>(lengths[b]) - after;
  if (at < 0 || at >= static_cast<long long>(table.max_pages) * c.page_size) {
    if (lane == 0) report(status, kDataLengthRange);
    return;
  }
  const int slot = static_cast<int>(at) / c.page_size;
  const int page = table.ids[b * table.stride + slot];
  if (page < 0 || page >= c.pages) {
    if (lane == 0) report(status, kDataPageRange);
    return;
  }
  const long long off = page * c.page_stride + (static_cast<int>(at) - slot * c.page_size) * c.token_stride;
  uint4* kd = reinterpret_cast<uint4*>(c.k + off) + lane;
  uint4* vd = reinterpret_cast<uint4*>(c.v + off) + lane;
  for (int j0 = 0;;) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (j0 + i * 32 + lane < vecs) {
        kd[j0 + i * 32] = kw[i];
        vd[j0 + i * 32] = vw[i];
      }
    if ((j0 += 32 * kPieces) >= vecs) break;
    load(j0);
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
                  ch.keep <= a.lengths[ch.parent] &&
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

// Workspace: refs[P], first[P] (cleared before the launch that counts in
// them), order[P] the free pages ascending, base[C] the first fresh
// rank of a sequence (sign bit: its last page stays), count of free pages.
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

// Sum of `mine`, one int a warp, over the warps before this one; `total` over
// all.
__device__ __forceinline__ int warps_before(int mine, int* scratch, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) scratch[warp] = mine;
  __syncthreads();
  const int x = scratch[lane];  // (32 warps)
  *total = __reduce_add_sync(0xffffffffu, x);
  return __reduce_add_sync(0xffffffffu, lane < warp ? x : 0);
}
static_assert(kPlanThreads == 32 * 32, "a lane a warp");

// A plan goes through the pages in rounds of kRun * 1024, a warp through kRun
// times 32 neighbours, a lane a page: what a lane ranks comes from ballots and
// one scan over the warps, and reads and writes are of neighbours.  (Eight
// neighbours a thread met bank conflicts and stores of 32 sectors: the plans'
// kernels took 12.5 us for a fork, 11.7 for a compaction, and take 9.8 and 8.2.)
constexpr int kRun = 8;
__device__ __forceinline__ int page_of_run(int p0, int i) {
  return p0 + (threadIdx.x >> 5) * (32 * kRun) + i * 32 + (threadIdx.x & 31);
}
__device__ __forceinline__ int lanes_before(unsigned int ballot) {
  return __popc(ballot & ((1u << (threadIdx.x & 31)) - 1u));
}

// From the counts (in shared or global memory): which last pages stay, every
// sequence's first fresh rank, the free pages and who is left.  One block.
__device__ void fork_plan(const ForkArgs& a, const ForkSpace& s, const int* refs, const int* first, int* scratch) {
  const int tid = threadIdx.x, P = a.cache.pages;
  int fresh_total = 0;
  for (int c0 = 0; c0 < a.C; c0 += kPlanThreads) {
    const int c = c0 + tid;
    int fresh = 0, stays = 0;
    if (c < a.C) {
      const Child ch = child_of(a, c);
      if (ch.tail > 0) {
        const int p = child_page(a, ch, ch.full);
        stays = p >= 0 && refs[p] == 0 && first[p] == a.C - c;
      }
      fresh = max(0, ch.need - ch.full - stays);
      a.new_lengths[c] = ch.keep;
    }
    int sum, incl = fresh;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if ((tid & 31) >= d) incl += o;
    }
    const int before = warps_before(__shfl_sync(0xffffffffu, incl, 31), scratch, &sum);
    if (c < a.C) s.base[c] = (fresh_total + before + incl - fresh) | (stays ? INT_MIN : 0);
    fresh_total += sum;
  }
  // the free pages ascending; the first of them are given out
  int before = 0;
  for (int p0 = 0; p0 < P; p0 += kPlanThreads * kRun) {
    int count[kRun], mine = 0;
    unsigned int free[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int p = page_of_run(p0, i);
      count[i] = p < P ? refs[p] : 1;
      if (count[i] == 0) count[i] = first[p] > 0;
      free[i] = __ballot_sync(0xffffffffu, count[i] == 0);
      mine += __popc(free[i]);
    }
    int sum;
    int rank = before + warps_before(mine, scratch, &sum);
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int p = page_of_run(p0, i), at = rank + lanes_before(free[i]);
      rank += __popc(free[i]);
      if (p >= P) continue;
      if (count[i] == 0) {
        s.order[at] = p;
        if (at >= fresh_total) a.free_pages[at - fresh_total] = p;
        else count[i] = 1;
      }
      a.ref_counts[p] = count[i];
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

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkArgs a, ForkSpace s) {
  __shared__ int scratch[32];
  fork_plan(a, s, s.refs, s.first, scratch);
}

// Writes the rows of the new table and copies the kept tokens of partly
// filled pages that did not stay: groups of threads take (sequence, table row
// or one layer's K or V).  (Shared out by 8 tokens, what every copy looks up
// first cost more than the evener shares gave: 28 us against 21 for 512
// sequences with 15 tokens each in 4 layers.)
__device__ void fork_write(const ForkArgs& a, const ForkSpace& s) {
  const CacheView& cv = a.cache;
  const int nfree = *s.nfree;
  const int vecs = cv.row_bytes() / 16, parts = 1 + 2 * cv.layers;
  const int lane = threadIdx.x % kGroup, groups = gridDim.x * (blockDim.x / kGroup);
  const long long items = static_cast<long long>(a.C) * parts;
  for (long long x = blockIdx.x * (blockDim.x / kGroup) + threadIdx.x / kGroup; x < items; x += groups) {
    const int c = static_cast<int>(x / parts), y = static_cast<int>(x - static_cast<long long>(c) * parts) - 1;
    const Child ch = child_of(a, c);
    const int packed = s.base[c], base = packed & INT_MAX;
    const int kept = ch.full + (packed < 0);
    if (y < 0) {
      int32_t* row = a.new_table + static_cast<long long>(c) * a.table.max_pages;
      for (int j = lane; j < a.table.max_pages; j += kGroup) {
        int p = -1;
        if (j < kept) p = child_page(a, ch, j);
        else if (j < ch.need && base + j - kept < nfree) p = s.order[base + j - kept];
        row[j] = p;
      }
    } else if (ch.tail > 0 && packed >= 0 && ch.full < ch.need && base < nfree) {
      const int from = child_page(a, ch, ch.full), to = s.order[base];
      if (from < 0) continue;
      char* pool = (y & 1 ? cv.v : cv.k) + (y >> 1) * cv.layer_stride;
      copy_tokens(cv, pool + from * cv.page_stride, pool + to * cv.page_stride, ch.tail, vecs, lane);
    }
  }
}

__global__ void __launch_bounds__(256) fork_write_kernel(const ForkArgs a, ForkSpace s) {
  after_plan();
  fork_write(a, s);
}

// Counts and plan by one block (10 us for 64 sequences of up to 1000 tokens, and
// for 8 parents of up to 250 pages and 512 sequences: dependent look-ups and
// scans).  The counts come by parent: ends[b][f]
// sequences keep f full pages of parent b, so page j of b gains the sum of
// ends[b][f] over f > j -- one addition a parent's page, however many
// sequences share it.
__global__ void __launch_bounds__(kPlanThreads, 1) fork_block_kernel(const ForkArgs a, ForkSpace s) {
  extern __shared__ int counts[];  // refs[P], first[P], ends[B][max_pages + 1]
  __shared__ int scratch[32];
  const int tid = threadIdx.x, lane = tid & 31, P = a.cache.pages, M = a.table.max_pages;
  int *refs = counts, *first = refs + P, *ends = first + P;
  const int words = 2 * P + a.B * (M + 1);
  for (int i = tid; i < words; i += kPlanThreads) counts[i] = 0;
  __syncthreads();
  int bad = 0;
  for (int c = tid; c < a.C; c += kPlanThreads) {
    const Child ch = child_of(a, c);
    bad |= ch.bad;
    if (ch.full > 0) atomicAdd(&ends[ch.parent * (M + 1) + ch.full], 1);
    if (ch.tail > 0) {
      const int p = child_page(a, ch, ch.full);
      if (p < 0) bad |= kDataPageRange;
      else atomicMax(&first[p], a.C - c);
    }
  }
  __syncthreads();
  // a warp a parent, its pages from the last to the first, four table entries a
  // lane on their way at once
  constexpr int kAhead = 4;
  for (int b = tid >> 5; b < a.B; b += kPlanThreads / 32) {
    const int S = a.cache.page_size, len = min(max(__ldg(a.lengths + b), 0), M * S);
    const int most = len / S;  // full pages that anyone can keep
    const int32_t* row = a.table.ids + b * a.table.stride;
    int beyond = 0;            // sequences that keep more than the pages seen so far
    for (int j0 = (most + 32 * kAhead - 1) / (32 * kAhead) * (32 * kAhead); j0 > 0;) {
      j0 -= 32 * kAhead;
      int page[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) page[i] = j0 + i * 32 + lane < most ? __ldg(row + j0 + i * 32 + lane) : 0;
#pragma unroll
      for (int i = kAhead - 1; i >= 0; --i) {
        if (j0 + i * 32 >= most) continue;
        const int j = j0 + i * 32 + lane;
        int sum = j < most ? ends[b * (M + 1) + j + 1] : 0;  // ends at j + 1: keeps page j
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_down_sync(0xffffffffu, sum, d);
          if (lane + d < 32) sum += o;
        }
        sum += beyond;
        if (j < most && sum > 0) {
          if (page[i] >= 0 && page[i] < P) atomicAdd(&refs[page[i]], sum);
          else bad |= kDataPageRange;
        }
        beyond = __shfl_sync(0xffffffffu, sum, 0);
      }
    }
  }
  report(a.status, bad);
  __syncthreads();
  fork_plan(a, s, refs, first, scratch);
}

// ---- compact -------------------------------------------------------------------
// Workspace: refs[P] (cleared before the launch that counts in them), to[P] the pages' new numbers, from[P] the moved pages ascending, holes[P], moves.
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

__device__ void compact_count(const CompactArgs& a, int* refs, int first, int step) {
  const long long entries = static_cast<long long>(a.B) * a.table.max_pages;
  int bad = 0;
  for (long long x = first; x < entries; x += step) {
    const int b = static_cast<int>(x / a.table.max_pages);
    const int p = a.table.ids[b * a.table.stride + (x - static_cast<long long>(b) * a.table.max_pages)];
    if (p >= a.cache.pages) bad = kDataPageRange;
    else if (p >= 0) atomicAdd(&refs[p], 1);
  }
  report(a.status, bad);
}

__global__ void __launch_bounds__(256) compact_count_kernel(const CompactArgs a, CompactSpace s) {
  compact_count(a, s.refs, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}

// From the counts: how many pages are in use, which move and where to.  One block.
__device__ void compact_plan(const CompactArgs& a, const CompactSpace& s, const int* refs, int* scratch) {
  const int tid = threadIdx.x, P = a.cache.pages;
  int mine = 0, n;
  for (int p = tid; p < P; p += kPlanThreads) mine += refs[p] > 0;
  warps_before(__reduce_add_sync(0xffffffffu, mine), scratch, &n);
  // movers (in use, at or above n) and holes (free, below n) in one scan, the
  // holes counted in the upper half
  static_assert(kPlanThreads * kRun < 1 << 15, "both fit");
  int moves = 0, holes = 0;
  for (int p0 = 0; p0 < P; p0 += kPlanThreads * kRun) {
    int count[kRun], both = 0;
    unsigned int mover[kRun], hole[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int p = page_of_run(p0, i);
      count[i] = p < P ? refs[p] : 0;
      mover[i] = __ballot_sync(0xffffffffu, count[i] > 0 && p >= n);
      hole[i] = __ballot_sync(0xffffffffu, p < min(n, P) && count[i] == 0);
      both += __popc(mover[i]) + (__popc(hole[i]) << 16);
    }
    int sum;
    const int start = warps_before(both, scratch, &sum);
    int at_m = moves + (start & 0xffff), at_h = holes + (start >> 16);
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int p = page_of_run(p0, i);
      const bool moves_it = count[i] > 0 && p >= n, is_hole = p < n && count[i] == 0;
      if (p < P) {
        if (moves_it) s.from[at_m + lanes_before(mover[i])] = p;
        else s.to[p] = p;
        if (is_hole) s.holes[at_h + lanes_before(hole[i])] = p;
        else a.ref_counts[p] = p < n ? count[i] : 0;
      }
      at_m += __popc(mover[i]);
      at_h += __popc(hole[i]);
    }
    moves += sum & 0xffff;
    holes += sum >> 16;
  }
  __syncthreads();
  for (int i = tid; i < moves; i += kPlanThreads) {
    const int from = s.from[i], to = s.holes[i];
    s.to[from] = to;
    a.ref_counts[to] = refs[from];
  }
  if (tid == 0) {
    *a.n_live = n;
    *s.moves = moves;
  }
}

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactArgs a, CompactSpace s) {
  __shared__ int scratch[32];
  compact_plan(a, s, s.refs, scratch);
}

// A group moves at most this many tokens of a page at a time, eight pieces a
// thread: whole pages (32 KB with 8 heads of 128) shared the work out less
// evenly (98 us against 97 for a pool of 4096 pages in 4 layers, half in use;
// now 91: the move alone is 78, its bytes at the copy rate 80, and the plan's
// block 8 comes before).
__host__ __device__ __forceinline__ int copy_chunk(const CacheView& cv) {
  const int vecs = static_cast<int>(cv.row_bytes() / 16);
  return vecs < 8 * kGroup ? 8 * kGroup / vecs : 1;
}
__host__ __device__ __forceinline__ int copy_chunks(const CacheView& cv) {
  const int n = copy_chunk(cv);
  return (cv.page_size + n - 1) / n;
}

// Rewrites the table and moves the pages: groups of threads take (page, some
// tokens of one layer's K or V).
__device__ void compact_move(const CompactArgs& a, const CompactSpace& s) {
  const CacheView& cv = a.cache;
  const int P = cv.pages;
  const long long entries = static_cast<long long>(a.B) * a.table.max_pages;
  for (long long x = blockIdx.x * blockDim.x + threadIdx.x; x < entries; x += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int b = static_cast<int>(x / a.table.max_pages);
    const int p = a.table.ids[b * a.table.stride + (x - static_cast<long long>(b) * a.table.max_pages)];
    a.new_table[x] = p >= 0 && p < P ? s.to[p] : -1;
  }
  const int moves = *s.moves, vecs = cv.row_bytes() / 16;
  const int chunk = copy_chunk(cv), chunks = copy_chunks(cv), parts = 2 * cv.layers * chunks;
  const int lane = threadIdx.x % kGroup, groups = gridDim.x * (blockDim.x / kGroup);
  const long long jobs = static_cast<long long>(moves) * parts;
  for (long long x = blockIdx.x * (blockDim.x / kGroup) + threadIdx.x / kGroup; x < jobs; x += groups) {
    const int i = static_cast<int>(x / parts), z = static_cast<int>(x - static_cast<long long>(i) * parts);
    const int y = z / chunks, t0 = (z - y * chunks) * chunk;
    const long long at = t0 * cv.token_stride;
    char* pool = (y & 1 ? cv.v : cv.k) + (y >> 1) * cv.layer_stride;
    copy_tokens(cv, pool + s.from[i] * cv.page_stride + at, pool + s.holes[i] * cv.page_stride + at,
                min(chunk, cv.page_size - t0), vecs, lane);
  }
}

__global__ void __launch_bounds__(256) compact_move_kernel(const CompactArgs a, CompactSpace s) {
  after_plan();
  compact_move(a, s);
}

__global__ void __launch_bounds__(kPlanThreads, 1) compact_block_kernel(const CompactArgs a, CompactSpace s) {
  extern __shared__ int counts[];  // refs[P]
  __shared__ int scratch[32];
  for (int i = threadIdx.x; i < a.cache.pages; i += kPlanThreads) counts[i] = 0;
  __syncthreads();
  // (as compact_count, four entries on their way at once, and in 32 bits)
  constexpr int kAhead = 4;
  const int entries = a.B * a.table.max_pages;
  int bad = 0;
  for (int x0 = threadIdx.x; x0 < entries; x0 += kAhead * kPlanThreads) {
    int page[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int x = x0 + i * kPlanThreads, b = x / a.table.max_pages;
      page[i] = x < entries ? __ldg(a.table.ids + b * a.table.stride + (x - b * a.table.max_pages)) : -1;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (page[i] >= a.cache.pages) bad = kDataPageRange;
      else if (page[i] >= 0) atomicAdd(&counts[page[i]], 1);
    }
  }
  report(a.status, bad);
  __syncthreads();
  compact_plan(a, s, counts, scratch);
}

// The copying kernel, as the dependent of the plan's.
template <typename A, typename S>
cudaError_t launch_after(void (*kernel)(A, S), const A& a, const S& s, long long groups, int sm_count, cudaStream_t stream) {
  const long long want = (groups * kGroup + 255) / 256;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned int>(want < 1 ? 1 : want < sm_count * 8 ? want : sm_count * 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, s);
}

size_t up(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

}  // namespace

cudaError_t launch_append(const char* k_new, const char* v_new, long long new_stride, int T,
                          const int32_t* starts, const CacheView& c, const PageTable& t,
                          const int32_t* lengths, int B, int32_t* status, cudaStream_t stream) {
  append_kernel<<<(T - 1) / 8 + 1, 256, 0, stream>>>(k_new, v_new, new_stride, T, starts, c, t, lengths, B, status);
  return cudaGetLastError();
}

cudaError_t cache_pages_prepare() {
  cudaError_t e = cudaFuncSetAttribute(fork_block_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(compact_block_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared);
  return e;
}

size_t fork_workspace(int pages, int C) {
  return up((3 * static_cast<size_t>(pages) + static_cast<size_t>(C) + 1) * 4);
}

cudaError_t launch_fork(const ForkArgs& a, void* ws, int sm_count, cudaStream_t stream) {
  const ForkSpace s = fork_space(ws, a.cache.pages, a.C);
  const long long words = 2ll * a.cache.pages + static_cast<long long>(a.B) * (a.table.max_pages + 1);
  if (words * 4 <= kMaxShared) {
    fork_block_kernel<<<1, kPlanThreads, static_cast<size_t>(words) * 4, stream>>>(a, s);
  } else {
    const cudaError_t e = cudaMemsetAsync(s.refs, 0, 2 * static_cast<size_t>(a.cache.pages) * 4, stream);
    if (e != cudaSuccess) return e;
    const int blocks = a.C < sm_count * 8 ? a.C : sm_count * 8;
    if (blocks > 0) fork_count_kernel<<<blocks, 256, 0, stream>>>(a, s);
    fork_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, s);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.C == 0) return e;
  return launch_after(fork_write_kernel, a, s, static_cast<long long>(a.C) * (1 + 2 * a.cache.layers), sm_count, stream);
}

size_t compact_workspace(int pages) { return up((4 * static_cast<size_t>(pages) + 1) * 4); }

cudaError_t launch_compact(const CompactArgs& a, void* ws, int sm_count, cudaStream_t stream) {
  const CompactSpace s = compact_space(ws, a.cache.pages);
  const long long entries = static_cast<long long>(a.B) * a.table.max_pages;
  const size_t smem = static_cast<size_t>(a.cache.pages) * 4;
  // (one block counts 64 Ki entries in less time than two more launches take)
  if (smem <= kMaxShared && entries <= (1 << 16)) {
    compact_block_kernel<<<1, kPlanThreads, smem, stream>>>(a, s);
  } else {
    const cudaError_t e = cudaMemsetAsync(s.refs, 0, smem, stream);
    if (e != cudaSuccess) return e;
    const long long want = (entries + 255) / 256;
    if (entries > 0)
      compact_count_kernel<<<static_cast<int>(want < sm_count * 8 ? want : sm_count * 8), 256, 0, stream>>>(a, s);
    compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, s);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long pieces = static_cast<long long>(a.cache.pages / 2) * 2 * a.cache.layers * copy_chunks(a.cache) + entries / kGroup;
  return launch_after(compact_move_kernel, a, s, pieces, sm_count, stream);
}

}  // namespace specv
