// attention_common.cuh -- how the paged attention kernels share out their
// work and join partial results (sm_103a).
//
// The rows of one cache head h of one sequence b are its Q queries times the
// G = Hq / heads query heads that read h, row = i * G + g; tiles of them are
// items (b, row tile, h).  An item's tokens are cut into tiles of a fixed
// number of tokens, and an item counts as its tiles and kEnd steps more, which
// is what its start and end cost (without them the block that gets a short
// sequence's items was last by a fifth: 64 sequences of 400..4000 tokens, six
// queries of 4 heads, 140 us against 114; one query 108 against 101).  The steps of all items are numbered item by item, and
// CTA c takes steps [c * per, (c + 1) * per).  So every CTA has the same work
// whatever the lengths are, and the cut is known without a word from the
// host, which does not see the lengths.  A CTA whose range holds only part of
// an item's tiles leaves (m, l, O) -- running maximum, sum and weighted sum --
// in its workspace slot; the item's last CTA to arrive joins the slots in CTA
// order, so the result does not depend on who was last.  When there is a CTA
// for every item and none has more than kWholeTiles tiles, nothing is cut: a
// join would take longer than those tiles (four sequences of 190 tokens in
// bf16: cut 14.7 us, whole 8.7).
#pragma once

#include "device_common.cuh"
#include "launch_decode.h"

namespace specv {

struct AttnPlan {
  long long total, per;  // steps in all, per CTA
  long long base;        // first step of sequence b
  int b;                 // sequence of the CTA's first step
  int pad;               // steps of every item, 0: its tiles and kEnd
};
constexpr int kWholeTiles = 8;

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
template <int kStep, int kEnd, int kThreadsA>
__device__ AttnPlan attn_plan(const AttnArgs& a, int items_per_seq, int min_tiles, long long* scratch) {
  constexpr int kW = kThreadsA / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (a.B + kThreadsA - 1) / kThreadsA;
  const int b0 = min(tid * run, a.B), b1 = min(b0 + run, a.B);
  long long mine = 0;
  int most = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const int n = attn_length(a, b), tiles = attn_tiles<kStep>(n);
    bad |= n != a.lengths[b];
    most = max(most, tiles);
    mine += tiles + kEnd;
  }
  if (bad && a.status && blockIdx.x == 0) atomicOr(a.status, kDataLengthRange);
  mine *= items_per_seq;
  most = __reduce_max_sync(0xffffffffu, most);
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) {
    scratch[warp] = incl;
    scratch[kW + 2 + warp] = most;
  }
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kW; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
    most = max(most, static_cast<int>(scratch[kW + 2 + w]));
  }
  AttnPlan p;
  if (most <= kWholeTiles && static_cast<long long>(a.B) * items_per_seq <= gridDim.x) {
    p.pad = most + kEnd;
    p.per = p.pad;
    p.total = static_cast<long long>(a.B) * items_per_seq * p.per;
    p.b = blockIdx.x / items_per_seq;
    p.base = static_cast<long long>(p.b) * items_per_seq * p.per;
    __syncthreads();
    return p;
  }
  incl += before;
  long long per = (total + gridDim.x - 1) / gridDim.x;
  if (per < min_tiles + kEnd) per = min_tiles + kEnd;
  const long long lo = per * blockIdx.x;
  if (lo >= incl - mine && lo < incl) {
    long long base = incl - mine;
    int b = b0;
    for (; b + 1 < b1; ++b) {
      const long long t = static_cast<long long>(attn_tiles<kStep>(attn_length(a, b)) + kEnd) * items_per_seq;
      if (lo < base + t) break;
      base += t;
    }
    scratch[kW] = b;
    scratch[kW + 1] = base;
  }
  __syncthreads();
  p.pad = 0;
  p.total = total;
  p.per = per;
  p.b = static_cast<int>(scratch[kW]);
  p.base = scratch[kW + 1];
  __syncthreads();
  return p;
}

// A CTA's parts of items, one after the other: next() gives tiles
// [tile0, tile1) of rows [row0, row0 + rows) of cache head h of sequence b.
template <int kStep, int kEnd, int kRows>
struct AttnWalk {
  const AttnArgs& a;
  long long w, end, per, base;
  int b, H, RT, R, pad;
  int n, tiles, size, item, tile0, tile1, used, rt, h, row0, rows;
  __device__ __forceinline__ AttnWalk(const AttnArgs& args, const AttnPlan& p) : a(args) {
    H = a.cache.heads;
    R = a.Q * (a.Hq / H);
    RT = (R + kRows - 1) / kRows;
    per = p.per;
    w = per * blockIdx.x;
    end = min(p.total, w + per);
    b = p.b;
    base = p.base;
    pad = p.pad;
    used = 0;
  }
  __device__ __forceinline__ bool next() {
    for (;;) {
      w += used;
      if (w >= end) return false;
      n = attn_length(a, b);
      tiles = attn_tiles<kStep>(n);
      size = pad ? pad : tiles + kEnd;
      while (w >= base + static_cast<long long>(size) * H * RT) {
        base += static_cast<long long>(size) * H * RT;
        n = attn_length(a, ++b);
        tiles = attn_tiles<kStep>(n);
        size = pad ? pad : tiles + kEnd;
      }
      item = static_cast<int>((w - base) / size);
      const int off = static_cast<int>((w - base) - static_cast<long long>(item) * size);
      const int stop = static_cast<int>(min(static_cast<long long>(size), off + (end - w)));
      used = stop - off;
      tile0 = max(off - kEnd, 0);  // an item's first kEnd steps are nobody's
      tile1 = min(stop - kEnd, tiles);
      if (tile0 < tile1) break;
    }
    rt = item / H;
    h = item - rt * H;
    row0 = rt * kRows;
    rows = min(kRows, R - row0);
    return true;
  }
  // step of the item's first tile
  __device__ __forceinline__ long long first() const { return base + static_cast<long long>(item) * size + kEnd; }
  __device__ __forceinline__ bool whole() const { return tile0 == 0 && tile1 == tiles; }
};

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

// Joins the parts of an item and writes its rows: a thread takes four
// dimensions of up to kE rows and adds the parts in CTA order.  The parts come
// from L2, some 600 cycles away, so the loads of kE rows and kC parts are under
// way together (one by one a join of two parts of 24 rows took 7 us).
template <int kRows, int D, int kThreadsA>
__device__ void attn_join(const AttnArgs& a, int b, int h, int row0, int rows, long long first, int tiles,
                          long long per) {
  constexpr int kEach = kRows * (D / 4) / kThreadsA, kE = kEach < 1 ? 1 : kEach < 3 ? kEach : 3, kC = 4;
  const long long c0 = first / per, c1 = (first + tiles - 1) / per;
  __threadfence();
  for (int e0 = threadIdx.x; e0 < rows * (D / 4); e0 += kE * kThreadsA) {
    int r[kE], d[kE];
    float m[kE], l[kE];
    float4 o[kE];
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      const int e = min(e0 + i * kThreadsA, rows * (D / 4) - 1);
      r[i] = e / (D / 4);
      d[i] = (e - r[i] * (D / 4)) * 4;
      m[i] = -INFINITY;
      l[i] = 0.f;
      o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (long long c = c0; c <= c1; c += kC) {
      float mc[kC][kE];
#pragma unroll
      for (int y = 0; y < kC; ++y)
#pragma unroll
        for (int i = 0; i < kE; ++i)
          mc[y][i] = __ldcg(attn_slot<kRows, D>(a, min(c + y, c1), min(c + y, c1) == c0) + kRows * D + r[i]);
#pragma unroll
      for (int y = 0; y < kC; ++y)
#pragma unroll
        for (int i = 0; i < kE; ++i) m[i] = fmaxf(m[i], mc[y][i]);
    }
    for (long long c = c0; c <= c1; c += kC) {
      float mc[kC][kE], lc[kC][kE];
      float4 v[kC][kE];
#pragma unroll
      for (int y = 0; y < kC; ++y) {
        const float* s = attn_slot<kRows, D>(a, min(c + y, c1), min(c + y, c1) == c0);
#pragma unroll
        for (int i = 0; i < kE; ++i) {
          mc[y][i] = c + y <= c1 ? __ldcg(s + kRows * D + r[i]) : -INFINITY;
          lc[y][i] = c + y <= c1 ? __ldcg(s + kRows * D + kRows + r[i]) : 0.f;
          v[y][i] = c + y <= c1 ? __ldcg(reinterpret_cast<const float4*>(s + r[i] * D + d[i])) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
#pragma unroll
      for (int y = 0; y < kC; ++y)
#pragma unroll
        for (int i = 0; i < kE; ++i) {
          // a part without a maximum holds zeros, or NaN that it passes on
          const float w = mc[y][i] == -INFINITY ? 1.f : ex2(mc[y][i] - m[i]);
          l[i] = fmaf(w, lc[y][i], l[i]);
          o[i].x = fmaf(w, v[y][i].x, o[i].x);
          o[i].y = fmaf(w, v[y][i].y, o[i].y);
          o[i].z = fmaf(w, v[y][i].z, o[i].z);
          o[i].w = fmaf(w, v[y][i].w, o[i].w);
        }
    }
#pragma unroll
    for (int i = 0; i < kE; ++i)
      if (e0 + i * kThreadsA < rows * (D / 4)) attn_write<D>(a, b, h, row0 + r[i], d[i], m[i], l[i], o[i]);
  }
}

}  // namespace specv
