// tree_common.cuh -- what a tree's nodes see of the tree (sm_103a).
//
// Node i sees its ancestors and itself: a bit set of up to kMaxNodes bits, made
// by following parents, which lie at lower indexes, so a walk ends.
#pragma once

#include "attention_common.cuh"
#include "device_common.cuh"
#include "launch_tree.h"

namespace specv {

// attention_common.cuh's plan of a call whose table has no room for more than
// kWholeTiles tiles a sequence, and whose items are no more than the blocks: the
// cut is known without the lengths (a block's scan of them takes 2 us).
template <int kEnd>
__device__ __forceinline__ AttnPlan attn_plan_whole(const AttnArgs& a, int items_per_seq) {
  AttnPlan p;
  p.b = blockIdx.x / items_per_seq;
  if (p.b < a.B && threadIdx.x == 0 && a.status && attn_length(a, p.b) != a.lengths[p.b]) atomicOr(a.status, kDataLengthRange);
  p.pad = kWholeTiles + kEnd;
  p.per = p.pad;
  p.total = static_cast<long long>(a.B) * items_per_seq * p.per;
  p.base = static_cast<long long>(p.b) * items_per_seq * p.per;
  return p;
}

// The bit sets of an item's rows.
template <int kRows>
struct TreeSight {
  int32_t parents[kMaxNodes];
  uint32_t bits[kRows][kNodeWords + 1];  // (the odd pitch spreads rows over the banks)
  uint8_t none[kRows];
  __device__ __forceinline__ bool sees(int row, int u) const { return (bits[row][(u >> 5) & (kNodeWords - 1)] >> (u & 31)) & 1; }
  // Bit y: does the row see token u0 + y, counted from the tree's first (those before it it does).
  __device__ __forceinline__ uint32_t window(int row, int u0) const {
    if (u0 <= -32) return 0xffffffffu;
    if (u0 < 0) return ((1u << -u0) - 1u) | (bits[row][0] << -u0);
    const int w = u0 >> 5;
    const uint32_t low = w < kNodeWords ? bits[row][w] : 0u, high = w + 1 < kNodeWords ? bits[row][w + 1] : 0u;
    return __funnelshift_r(low, high, u0);
  }
  __device__ __forceinline__ bool blind(int row) const { return none[row] != 0; }
};
template <>
struct TreeSight<0> {};

// Fills `sight` for rows row0, row0 + 1, ... of a cache head (row = node * G + query
// head of the group; those behind row `last` are as it) of sequence b, whose
// tree starts at token `base`, by `count` threads that `sync` holds together.
template <int kRows, typename Sync>
__device__ __forceinline__ void tree_sight(const AttnArgs& a, int b, int base, int row0, int last, int tid, int count,
                                           TreeSight<kRows>& sight, Sync sync) {
  const int32_t* parents = a.parents + b * a.parents_stride;
  bool bad = false;
#pragma unroll 1
  for (int i = tid; i < a.Q; i += count) {
    const int p = __ldg(parents + i);
    bad |= p >= i;
    sight.parents[i] = p;
  }
  if (bad && a.status) atomicOr(a.status, kDataTreeParent);
  sync();
  const int G = a.Hq / a.cache.heads;
#pragma unroll 1
  for (int r = tid; r < kRows; r += count) {
    const int node = min(row0 + r, last) / G;
    uint32_t* bits = sight.bits[r];
#pragma unroll
    for (int x = 0; x < kNodeWords; ++x) bits[x] = 0;
    // up the line, a word's bits gathered before they are stored (parents lie lower)
    int i = node, p;
    uint32_t word = 0;
#pragma unroll 1
    for (;;) {
      word |= 1u << (i & 31);
      p = sight.parents[i];
      const bool up = p >= 0 && p < i;
      if (!up || (p >> 5) != (i >> 5)) {
        bits[i >> 5] = word;
        word = 0;
      }
      if (!up) break;
      i = p;
    }
    sight.none[r] = p != -1 || base + node < 0;
  }
  sync();
}

}  // namespace specv
