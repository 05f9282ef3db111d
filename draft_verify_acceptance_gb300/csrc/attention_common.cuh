// attention_common.cuh -- how the paged attention kernels share out their
// work and join partial results (sm_103a).
//
// The rows of one cache head h of one sequence b are its Q queries times the
// G = Hq / heads query heads that read h, row = i * G + g; tiles of them are
// items (b, row tile, h).  An item's tokens are cut into steps of a fixed
// number of tokens, the steps of all items are numbered item by item, and
// CTA c takes steps [c * per, (c + 1) * per).  So every CTA has the same
// work whatever the lengths are, and the cut is known without a word from
// the host, which does not see the lengths.  A CTA whose range holds only
// part of an item leaves (m, l, O) -- running maximum, sum and weighted sum
// -- in its workspace slot; the item's last CTA to arrive joins the slots in
// CTA order, so the result does not depend on who was last.
#pragma once

#include "device_common.cuh"
#include "launch_decode.h"

namespace specv {

struct AttnPlan {
  long long total, per;  // steps in all, per CTA
  long long base;        // first step of sequence b
  int b;                 // sequence of the CTA's first step
};

__device__ __forceinline__ int attn_length(const AttnArgs& a, int b) {
  const int most = a.table.max_pages * a.cache.page_size;
  return min(max(a.lengths[b], 0), most);
}

// Steps of a sequence's items: an empty sequence still has one, which writes
// its rows.
template <int kStep>
__device__ __forceinline__ int attn_tiles(int n) {
  return max(1, (n + kStep - 1) / kStep);
}

// The cut, computed by every CTA from the lengths: each thread sums a run of
// sequences, the runs are scanned, and the thread whose run holds the CTA's
// first step walks it.  `scratch`: 2 * blockDim/32 + 4 long longs of shared
// memory.
template <int kStep, int kThreadsA>
__device__ AttnPlan attn_plan(const AttnArgs& a, int items_per_seq, int min_per,
                              long long* scratch) {
  constexpr int kW = kThreadsA / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (a.B + kThreadsA - 1) / kThreadsA;
  const int b0 = min(tid * run, a.B), b1 = min(b0 + run, a.B);
  long long mine = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const int n = attn_length(a, b);
    bad |= n != a.lengths[b];
    mine += attn_tiles<kStep>(n);
  }
  if (bad && a.status && blockIdx.x == 0) atomicOr(a.status, kDataLengthRange);
  mine *= items_per_seq;
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kW; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  incl += before;
  long long per = (total + gridDim.x - 1) / gridDim.x;
  if (per < min_per) per = min_per;
  const long long lo = per * blockIdx.x;
  if (lo >= incl - mine && lo < incl) {
    long long base = incl - mine;
    int b = b0;
    for (; b + 1 < b1; ++b) {
      const long long t = static_cast<long long>(attn_tiles<kStep>(attn_length(a, b))) * items_per_seq;
      if (lo < base + t) break;
      base += t;
    }
    scratch[kW] = b;
    scratch[kW + 1] = base;
  }
  __syncthreads();
  AttnPlan p;
  p.total = total;
  p.per = per;
  p.b = static_cast<int>(scratch[kW]);
  p.base = scratch[kW + 1];
  __syncthreads();
  return p;
}

// Where the CTA left part of an item: slot 1 of a CTA for the item that
// starts in its range, slot 0 for one that started before it.
template <int kRows, int D>
__device__ __forceinline__ float* attn_slot(const AttnArgs& a, long long cta, int which) {
  return a.partials + (cta * 2 + which) * (kRows * (D + 2));
}

// Row `row` of item (b, h): its query and query head.
struct AttnRow {
  int i, hq;
};
__device__ __forceinline__ AttnRow attn_row(const AttnArgs& a, int row, int h) {
  const int G = a.Hq / a.cache.heads;
  AttnRow r;
  r.i = row / G;
  r.hq = h * G + (row - r.i * G);
  return r;
}

__device__ __forceinline__ void store4(void* out, size_t at, bool bf16, float4 v) {
  if (bf16) {
    uint2 w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(v.y), "f"(v.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(v.w), "f"(v.z));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = w;
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = v;
  }
}

constexpr float kLn2 = 0.693147181f;

// Four dimensions of a finished row: out = O / l, and for the first of them
// lse = (m + log2 l) ln 2 (m in units of log2).
template <int D>
__device__ __forceinline__ void attn_write(const AttnArgs& a, int b, int h, int row, int d, float m,
                                           float l, float4 o) {
  const AttnRow r = attn_row(a, row, h);
  const size_t at = (static_cast<size_t>(b) * a.Q + r.i) * a.Hq + r.hq;
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  o.x *= inv;
  o.y *= inv;
  o.z *= inv;
  o.w *= inv;
  store4(a.out, at * D + d, a.cache.bf16, o);
  if (d == 0 && a.lse) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Counts this CTA's part of the item whose steps are [first, first + tiles);
// true for the whole block in the CTA that came last, which then joins.
__device__ __forceinline__ bool attn_arrive(const AttnArgs& a, long long first, int tiles, long long per,
                                            int* flag) {
  __syncthreads();  // the block's stores to its slot are done
  if (threadIdx.x == 0) {
    const long long c0 = first / per, c1 = (first + tiles - 1) / per;
    const unsigned int n = static_cast<unsigned int>(c1 - c0 + 1);
    __threadfence();
    const bool last = atom_add_acq_rel_gpu(&a.counters[c0], 1u) + 1u == n;
    if (last) a.counters[c0] = 0u;
    *flag = last;
  }
  __syncthreads();
  return *flag != 0;
}

// Joins the parts of an item and writes its rows: thread by thread four
// dimensions of a row, over the parts in CTA order.
template <int kRows, int D, int kThreadsA>
__device__ void attn_join(const AttnArgs& a, int b, int h, int row0, int rows, long long first, int tiles,
                          long long per) {
  const long long c0 = first / per, c1 = (first + tiles - 1) / per;
  __threadfence();
  for (int e = threadIdx.x; e < rows * (D / 4); e += kThreadsA) {
    const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
    float m = -INFINITY;
    for (long long c = c0; c <= c1; ++c)
      m = fmaxf(m, __ldcg(attn_slot<kRows, D>(a, c, c == c0) + kRows * D + r));
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (long long c = c0; c <= c1; ++c) {
      const float* s = attn_slot<kRows, D>(a, c, c == c0);
      const float mc = __ldcg(s + kRows * D + r);
      const float w = mc == -INFINITY ? 0.f : ex2(mc - m);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(s + r * D + d));
      l = fmaf(w, __ldcg(s + kRows * D + kRows + r), l);
      o.x = fmaf(w, v.x, o.x);
      o.y = fmaf(w, v.y, o.y);
      o.z = fmaf(w, v.z, o.z);
      o.w = fmaf(w, v.w, o.w);
    }
    attn_write<D>(a, b, h, row0 + r, d, m, l, o);
  }
}

}  // namespace specv
