// attention_tree_tc.cuh -- bf16 attention of trees with more than a few rows a
// cache head, on tcgen05 (sm_103a).
//
// Rows (nodes times query heads of a group) take the tensor cores' 128 lanes:
//     S [128 rows x 64 tokens] = Q K^T     A = Q, B = K, both from shared memory
//     O [128 rows x D]        += P V       A = P from TMEM, B = V as it lies
// so that a softmax thread holds one row, and its maximum, sum and rescaling
// need no word from another thread.  P takes the place of S in TMEM as two bf16
// parts (hi and lo, 2^-17 of a weight: one part would lose as much as rounding the
// output does).
//
// Two streams of such products run in turn, each with its softmax warps, two
// S / P buffers and an O of its own, so that one's products run under the other's
// softmax:  kDual, more than 128 rows: a stream for each 128 of an item's 256 rows,
// both over every tile;  else one for the even tiles and one for the odd ones,
// joined at the item's end.
//
// One block per SM.  Warps 0-3 and 4-7: the streams' softmax.  Warps 8-11 copy K
// and V of the tiles into a ring of slots, across item boundaries, in 16-byte
// pieces that arrive on the slot's barrier by themselves, so any page size and
// strides.  Warp 12 issues the scores' products, warp 13 the outputs'.
//
// Parts of an item that blocks' ranges cut are left in the workspace and joined by
// a dependent kernel over all SMs, in block order (one block would have to read
// up to 133 KB a part).
//
// The code is kept short: with loops unrolled to 200 KB the roles evicted each
// other from the instruction caches, and a tile took 4000 cycles.
//
// 32 query heads of 128 on 8 (ranges are over machines and lengths):  64 sequences of
// 400..4000 tokens, 16 nodes (64 rows a head) 108 to 117 us (the cache's bytes at the copy
// rate: 87; a block's tile 1300 cycles, an item's start and end 5 us of a block's time, part of it
// hidden behind the ring);  2 of 60001..131072, 26 nodes: 153 to 187 us (124 to 148);  32 of
// 400..4000, 64 nodes (256 rows): 102 to 113 us (45), a tile 2300 cycles of products, the
// scores' as long as the outputs' since each reads 4 KB of queries for 64 tokens;  the same
// with 33 nodes (132 rows) 103 and with 65 (260 rows: two items, the second nearly empty) 189;  one
// of 2111, 60 nodes: 25 us, start, part and join.  32 of 400..4000 over heads of 64, 30 nodes:
// 56 us (23), by the softmax's latency.
#pragma once

#include "attention_common.cuh"
#include "attention_mma.cuh"
#include "attention_tc.cuh"
#include "tree_common.cuh"

#include <type_traits>

namespace specv {
namespace ttc {

using mma::cp16;
using mma::nonfinite2;
using mma::pack2;
using tc::async_fence;
using tc::cp_arrive;
using tc::operand;
using tc::tc_after;
using tc::tc_before;
using tc::tc_commit;
using tc::tmem_alloc;
using tc::tmem_free;
using tc::tmem_st_done;

constexpr int kTile = 64;        // tokens
constexpr int kSoft = 256;       // softmax threads, 128 a stream
constexpr int kLoadWarps = 4;    // K and V of the even and of the odd tiles
constexpr int kThreadsR = kSoft + kLoadWarps * 32 + 128;
// Registers a thread: 512 x 128 at the launch, then shared out by groups of four
// warps, 2 x 128 x (176 + 80) = 512 x 128.
constexpr int kSoftRegs = 176, kOtherRegs = 80;
static_assert(kSoft * kSoftRegs + (kThreadsR - kSoft) * kOtherRegs <= 65536 && kThreadsR * 128 <= 65536, "registers");
constexpr int kScores = 8 + kLoadWarps, kOutputs = kScores + 1;   // the warps that issue products,
constexpr int kWalker = kOutputs + 1, kQueries = kWalker + 1;     // the one that finds the block's items, the one that copies queries
constexpr float kSlackR = 8.f;   // how far (log2) a score may pass the reference
// Steps that an item's start and end count as (two row tiles; one).  4 and 6: 64 x 16
// nodes over 400..4000 tokens 112.8 us, 32 x 64 110.9, 20 x 40 over 100..1500 42.9;  5 and
// 8: 113.0, 111.3, 43.9;  6 and 10: 114.8, 112.1, 44.2.
template <bool kDual>
constexpr int kEndR = kDual ? 4 : 6;
// Steps that a block gets at least, when there are more blocks than work: an item of T
// tiles cut into parts of p takes p tiles, and T / p parts to join, so p goes with the
// root of T.  One tree, one row tile: T = 11, 3 and 4 steps 17 us, 6 and 8 18.7, 12 20.7;
// T = 32, 4 21.6, 6 20.6, 8 21.2, 12 22.6;  T = 125, 7 30.8, 8 29.0, 12 27.1.  Two row tiles:
// T = 16 (two trees), 2 to 4 22.6, 6 24.7;  T = 33, 2 27.2, 4 24.7, 6 26.5.
template <bool kDual>
constexpr float kLeast = kDual ? 0.7f : 1.f;  // times the root of the most tiles
constexpr int kMaxCtas = 160;
constexpr int kAhead = 32;       // tiles whose valid bits are kept, more than the ring holds
constexpr int kOdd = 8;          // items whose flag is kept, more than a stream can be behind

template <int D, bool kDual>
struct Lay {
  static constexpr int kRows = kDual ? 256 : 128;  // of an item
  static constexpr int kSlot = kTile * D * 2;      // K or V of a tile
  static constexpr int kHalf = kTile * 128;        // 64 dimensions of it
  static constexpr int kQ = kRows * D * 2;
  static constexpr int kSlots = (227 * 1024 - 17 * 1024 - kQ) / kSlot;
  static constexpr int kBytes = kSlots * kSlot + kQ + 1024;  // 1024: alignment (some 15 KB more are static)
  static_assert(kSlots >= 8 && kSlots / 2 + 4 < kAhead, "the ring");
};

// An item, or this block's part of it.  One warp finds them for the others (the
// walk takes some thousand cycles an item, and a third of the softmax warps' registers).
struct Item {
  int any;   // 0: there are no more
  int end;   // block that has its last tile
  int b, h, n, rt, row0, rows, tile0, tile1, tiles;
  __device__ __forceinline__ bool whole() const { return tile0 == 0 && tile1 == tiles; }
};
// Kept: the softmax warps' own, kHeld - 1 before it, the rest told ahead, of one tile each as
// many as the ring and the loaders' look-ups are ahead (400 trees of 7 nodes over
// 10..60 tokens, heads of 64: 16 83 us, 8 89; others the same).
constexpr int kItems = 16;
constexpr int kHeld = 2;   // items that the softmax warps start before the first of them is given up

// What the host divides for the kernel (32-bit divisions take some 140 cycles, 64-bit ones 500).
struct Shape {
  int G, R, RT;  // query heads of a cache head, rows of one (nodes times G), items that they make
  DivU64 by_page, by_group, by_heads, by_items;  // page_size, G, cache heads, items of a sequence
};
__device__ __forceinline__ AttnRow row_of(const Shape& z, int row, int h) {
  AttnRow r;
  r.i = static_cast<int>(z.by_group(static_cast<unsigned long long>(row)));
  r.hq = h * z.G + (row - r.i * z.G);
  return r;
}

// One warp's walk over the items of its block, after attention_common.cuh's cut:
// an item's tiles and kEnd steps more are numbered item by item, sequence by
// sequence, and block c takes steps [c * per, (c + 1) * per).  With a block for every
// item and none of more than kWholeTiles tiles, nothing is cut.
template <int kRows, int kEnd>
struct Walker {
  const AttnArgs& a;
  long long w, end, per, base;  // step, last step and number of steps of the block; first step of sequence b
  const Shape& z;
  int lane, b, H, RT, n, tiles;
  bool whole;
  // (64 bits take this GPU 500 cycles and much code)
  __device__ __noinline__ static long long divide64(long long x, long long y) { return x / y; }
  __device__ __forceinline__ static long long divide(long long x, long long y) {
    if ((x | y) >> 32) return divide64(x, y);
    return static_cast<unsigned>(x) / static_cast<unsigned>(y);
  }
  __device__ __forceinline__ void sequence() {
    n = attn_length(a, b);
    tiles = attn_tiles<kTile>(n);
  }
  __device__ Walker(const AttnArgs& args, const Shape& shape, int lane_) : a(args), z(shape), lane(lane_) {
    H = a.cache.heads;
    RT = z.RT;
    long long total = 0;
    int most = 0;
    bool bad = false;
    const long long items = static_cast<long long>(a.B) * H * RT;
    if (a.whole) {  // (the lengths' scan takes 2 us)
      const int own = static_cast<int>(z.by_items(blockIdx.x));
      if (own < a.B) bad = attn_length(a, own) != a.lengths[own];
      if (bad && a.status && lane == 0) atomicOr(a.status, kDataLengthRange);
    }
#pragma unroll 1
    for (int i = a.whole ? a.B : lane; i < a.B; i += 32) {
      const int len = attn_length(a, i), t = attn_tiles<kTile>(len);
      bad |= len != a.lengths[i];
      most = max(most, t);
      total += t + kEnd;
    }
    if (!a.whole && bad && a.status && blockIdx.x == 0) atomicOr(a.status, kDataLengthRange);
    most = __reduce_max_sync(0xffffffffu, most);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    total *= H * RT;
    whole = most <= kWholeTiles && items <= gridDim.x;  // (a.whole: most is 0)
    if (whole) {
      w = blockIdx.x;
      end = items;
      b = static_cast<int>(z.by_items(blockIdx.x));
      base = static_cast<long long>(b) * H * RT;
      if (w < end) sequence();
      return;
    }
    per = divide(total + gridDim.x - 1, gridDim.x);
    per = max(per, static_cast<long long>(fmaf(kRows == 256 ? kLeast<true> : kLeast<false>, sqrtf(static_cast<float>(most)), 0.5f)));
    w = per * blockIdx.x;
    end = min(total, w + per);
    // the sequence that has step w, 32 sequences at a time
    base = 0;
    b = 0;
    if (w >= end) return;
#pragma unroll 1
    for (int i0 = 0;; i0 += 32) {
      const long long mine = i0 + lane < a.B ? static_cast<long long>(attn_tiles<kTile>(attn_length(a, i0 + lane)) + kEnd) * (H * RT) : 0;
      long long upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, w < base + upto);
      if (past) {
        const int l = __ffs(past) - 1;
        b = i0 + l;
        base += __shfl_sync(0xffffffffu, upto - mine, l);
        break;
      }
      base += __shfl_sync(0xffffffffu, upto, 31);
    }
    sequence();
  }
  __device__ void next(Item& i) {
    for (;;) {
      i.any = w < end;
      if (!i.any) return;
      const int size = whole ? 1 : tiles + kEnd;
      if (w >= base + static_cast<long long>(size) * H * RT) {
        base += static_cast<long long>(size) * H * RT;
        ++b;
        sequence();
        continue;
      }
      const long long in = w - base;
      const int item = static_cast<int>(divide(in, size)), off = static_cast<int>(in - static_cast<long long>(item) * size);
      const int stop = whole ? 1 : static_cast<int>(min(static_cast<long long>(size), off + (end - w)));
      i.tile0 = whole ? 0 : max(off - kEnd, 0);  // an item's first kEnd steps are nobody's
      i.tile1 = whole ? tiles : min(stop - kEnd, tiles);
      const long long first = base + static_cast<long long>(item) * size + kEnd;  // step of the item's first tile
      w = whole ? end : w + (stop - off);
      if (i.tile0 >= i.tile1) continue;
      i.tiles = tiles;
      i.n = n;
      i.b = b;
      i.rt = static_cast<int>(z.by_heads(static_cast<unsigned long long>(item)));
      i.h = item - i.rt * H;
      i.row0 = i.rt * kRows;
      i.rows = min(kRows, z.R - i.row0);
      i.end = i.whole() ? 0 : static_cast<int>(divide(first + tiles - 1, per));
      return;
    }
  }
};

// The item whose first tile a block has and whose last one another block; rows 0:
// there is none.
struct __align__(8) Join {
  int b, h, row0, rows, end, pad;
};

template <int D, bool kDual>
struct Shared {
  unsigned long long full[Lay<D, kDual>::kSlots], empty[Lay<D, kDual>::kSlots];
  unsigned long long s_full[2][2], p_full[2][2], pv_done[2][2], q_full, q_free, done[2];
  unsigned long long item_ready[kItems], item_free[kItems];
  Item item[kItems], none;
  uint2 valid[kAhead];  // tokens that exist, by tile
  TreeSight<128> sight[2];
  float m[2][128], l[2][128];
  int odd[kOdd];              // the item has values that are not finite and not every row sees
  uint32_t tmem;
  int dead;                   // a wait ran out: nothing waits any more
};

// The products of a tile, issued by one lane in one go (a product of its own, with
// its election and its descriptors, took ten instructions).
// S = Q K^T: steps of 16 dimensions, 64 a half of the operands.
template <int D>
__device__ __forceinline__ void scores_mma(uint32_t d, uint64_t a, uint64_t b) {
  constexpr uint32_t kKind = tc::instruction<kTile>(false, false);
  if constexpr (D == 128)
    asm volatile(
        "{\n\t.reg .pred p, q, e;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, 0, 0;\n\tsetp.eq.u32 q, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
        "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
        "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
        "add.s64 a, %1, 1024;\n\tadd.s64 b, %2, 512;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
        "add.s64 a, %1, 1026;\n\tadd.s64 b, %2, 514;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
        "add.s64 a, %1, 1028;\n\tadd.s64 b, %2, 516;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
        "add.s64 a, %1, 1030;\n\tadd.s64 b, %2, 518;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(kKind)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q, e;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, 0, 0;\n\tsetp.eq.u32 q, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
        "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
        "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(kKind)
        : "memory");
}
// O += P V: steps of 16 tokens; P lies as hi, lo of 32 tokens, hi, lo of the other 32.
template <int D>
__device__ __forceinline__ void outputs_mma(uint32_t d, uint32_t p, uint64_t v, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q, e;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.eq.u32 q, 0, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.s32 a, %1, 16;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], %2, %3, q;\n\t"
      "add.s64 b, %2, 128;\n\t"
      "add.s32 a, %1, 8;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t"
      "add.s32 a, %1, 24;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t"
      "add.s64 b, %2, 256;\n\t"
      "add.s32 a, %1, 32;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t"
      "add.s32 a, %1, 48;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t"
      "add.s64 b, %2, 384;\n\t"
      "add.s32 a, %1, 40;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t"
      "add.s32 a, %1, 56;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t}" ::"r"(d),
      "r"(p), "l"(v), "r"(tc::instruction<D>(false, true)), "r"(add ? 1u : 0u)
      : "memory");
}
#define SPEC_R8(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]), "=r"(x[i + 5]), "=r"(x[i + 6]), "=r"(x[i + 7])
#define SPEC_I8(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])
// Columns of the warp's lanes (the wait in the same statement: no use comes before it).
__device__ __forceinline__ void ld32(uint32_t (&r)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
      : SPEC_R8(r, 0), SPEC_R8(r, 8), SPEC_R8(r, 16), SPEC_R8(r, 24)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void ld64(uint32_t (&r)[64], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,"
      "%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\ttcgen05.wait::ld.sync.aligned;"
      : SPEC_R8(r, 0), SPEC_R8(r, 8), SPEC_R8(r, 16), SPEC_R8(r, 24), SPEC_R8(r, 32), SPEC_R8(r, 40), SPEC_R8(r, 48), SPEC_R8(r, 56)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void ld16(uint32_t (&r)[16], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : SPEC_R8(r, 0), SPEC_R8(r, 8)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::SPEC_I8(r, 0),
      SPEC_I8(r, 8), "r"(at)
      : "memory");
}
#undef SPEC_R8
#undef SPEC_I8

// Two fp32 operations at a time.
__device__ __forceinline__ uint64_t pair(uint32_t x, uint32_t y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(x), "r"(y));
  return d;
}
__device__ __forceinline__ void split(uint64_t d, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(d)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ void stream_sync(int s) { asm volatile("bar.sync %0, 128;" ::"r"(3 + s) : "memory"); }

// 16 bytes of the cache (0: zeros), with an L2 policy.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes, unsigned long long policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::256B [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes),
               "l"(policy)
               : "memory");
}
// What is read once makes room first (partial results and page tables stay: 64 x 16
// nodes 112.1 -> 108.0 us, long sequences 161 -> 155).
__device__ __forceinline__ unsigned long long policy_of(bool once) {
  unsigned long long p;
  if (once) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// Is x true in one of `count` threads of barrier `id`.
__device__ __forceinline__ bool any_of(int id, int count, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "r"(id), "r"(count)
      : "memory");
  return r != 0;
}

template <int D, bool kDual>
__global__ void __launch_bounds__(kThreadsR, 1) attention_tree_kernel(const AttnArgs a, const Shape z, Join* joins) {
  using L = Lay<D, kDual>;
  constexpr int kSlots = L::kSlots, kHalf = L::kHalf, kChunks = D / 8;  // 16-byte pieces of a token
  constexpr int kCols = 512, kStream = 256, kO = 128;                   // TMEM: a stream's S / P buffers, then its O
  extern __shared__ char raw_smem[];
  __shared__ Shared<D, kDual> sh;
  char* smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  char* q_s = smem + kSlots * L::kSlot;  // [128-row tiles][halves][128][128 bytes]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // (short: it stands in many places, and the roles' code shares the instruction caches)
  auto wait = [&](unsigned long long* bar, uint32_t parity) {
    int polls = 1 << 16;
#ifdef SPEC_DEBUG
    // (a test's way to a wait that ran out: a bit of the status word that it passes)
    if (blockIdx.x == 0 && a.status && (*reinterpret_cast<volatile int32_t*>(a.status) >> 30) != 0) {
      *reinterpret_cast<volatile int*>(&sh.dead) = 1;
      return;
    }
#endif
#pragma unroll 1
    while (!mbar_try_wait_sleep(bar, parity, 20000u))
      if (--polls == 0 || *reinterpret_cast<volatile int*>(&sh.dead)) {
        *reinterpret_cast<volatile int*>(&sh.dead) = 1;
        break;
      }
  };

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) joins[blockIdx.x] = {0, 0, 0, 0, 0, 0};
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sh.full[i], 33);
      mbar_init(&sh.empty[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sh.s_full[s][i], 1);
        mbar_init(&sh.p_full[s][i], 4);
        mbar_init(&sh.pv_done[s][i], 1);
      }
      mbar_init(&sh.done[s], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&sh.item_ready[i], 1);
      mbar_init(&sh.item_free[i], 2);
    }
    mbar_init(&sh.q_full, L::kRows);
    mbar_init(&sh.q_free, 1);
    for (int i = 0; i < kOdd; ++i) sh.odd[i] = 0;
    sh.dead = 0;
    sh.none.any = 0;
    fence_barrier_init();
  }
  if (warp == kOutputs) tmem_alloc(&sh.tmem, kCols);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = sh.tmem;

  auto item = [&](int k) -> const Item& {
    wait(&sh.item_ready[k % kItems], (k / kItems) & 1);
    return *reinterpret_cast<volatile int*>(&sh.dead) ? sh.none : sh.item[k % kItems];  // (one that was not told has no end)
  };

  // Copies 32 rows of an item's queries; behind the last row come zeros.
  auto load_q = [&](const Item& at, int y) {
    constexpr int kStep = 32 / kChunks;
    const int rows = at.rows, chunk = lane % kChunks, r0 = lane / kChunks;
    const AttnRow ar = row_of(z, at.row0 + min(y * 32 + lane, rows - 1), at.h);
    const long long off = at.b * a.q_batch + ar.i * a.q_token + ar.hq * a.q_head;
    const uint32_t to = smem_addr(q_s) + (y >> 2) * (128 * D * 2) + (chunk >> 3) * (128 * 128) + ((y & 3) * 32 + r0) * 128;
#pragma unroll 4
    for (int i = 0; i < 32; i += kStep)
      cp16(to + i * 128 + (((chunk & 7) ^ ((i + r0) & 7)) << 4), a.q + __shfl_sync(0xffffffffu, off, i + r0) + chunk * 16,
           y * 32 + i + r0 < rows ? 16 : 0);
    cp_arrive(&sh.q_full);
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
#ifdef SPEC_DEBUG
    // (another bit: the warps that a block's first item may need nothing of are a millisecond late)
    if ((warp == kQueries || warp == 10 || warp == 11) && a.status && (*reinterpret_cast<volatile int32_t*>(a.status) >> 29 & 1))
      for (int i = 0; i < 1000; ++i) __nanosleep(1000);
#endif
    if (warp < kScores) {
      // ---- K and V of each tile, in turn -----------------------------------
      // A warp takes K or V of every other tile, so that it looks its 64 tokens up
      // and waits once for 32 copies (with 16 tokens of every K and V a warp these
      // took more of its time than the copies).
      const bool is_v = warp & 1;
      const unsigned long long policy = policy_of(z.RT == 1);  // (more row tiles read the cache again)
      const int S = a.cache.page_size, chunk = lane % kChunks, r0 = lane / kChunks;
      constexpr int kStep = 32 / kChunks, kPasses = 8 / kStep;
      const bool in_page = S % 8 == 0;  // tokens 8 g .. 8 g + 7 of a tile lie in one page
      // The pages of tokens lane and 32 + lane, looked up a tile of the warp's ahead:
      // the table's entries are on their way while the tiles before are copied.
      struct Pages {
        int page[2], place[2], head;  // place: token in the page, -1: past the end
        bool any;
      } now = {}, next = {};
      int items = -1, tile = 0, tile1 = 0, n = 0, head = 0;
      int ahead = warp < 10 ? 1 : 2;  // tiles to go on by: the second pair starts with the second
      bool more = true;
      const int32_t* ids = nullptr;
      auto look_up = [&]() {
#pragma unroll 1
        for (; more && ahead > 0; --ahead) {
          if (++tile < tile1) continue;
          const Item& at = item(++items);
          more = at.any;
          tile = at.tile0;
          tile1 = at.tile1;
          n = at.n;
          head = at.h;
          ids = a.table.ids + at.b * a.table.stride;
        }
        ahead = 2;
        next.any = more;
        if (!more) return;
        next.head = head;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int t = tile * kTile + y * 32 + lane;
          const int entry = static_cast<int>(z.by_page(static_cast<unsigned long long>(t)));
          next.place[y] = t < n ? t - entry * S : -1;
          next.page[y] = t < n ? __ldg(ids + entry) : -1;
        }
      };
      const uint32_t ring = smem_addr(smem) + (chunk >> 3) * kHalf + r0 * 128;
      const char* pool = (is_v ? a.cache.v : a.cache.k) + chunk * 16 + r0 * a.cache.token_stride;
      const long long stride = kStep * a.cache.token_stride;
      int slot = warp - 8;
      uint32_t turn = 1;  // the parity of a slot that is free the first time
#pragma unroll 1
      for (int tile_no = ((warp - 8) >> 1) - 4; tile_no < 0 || now.any; tile_no += 2) {  // (two rounds fill `now` and `next`)
        uint32_t exist[2];
        long long off[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const bool ok = now.page[y] >= 0 && now.page[y] < a.cache.pages;
          if (!ok && now.place[y] >= 0 && tile_no >= 0 && a.status) atomicOr(a.status, kDataPageRange);
          exist[y] = __ballot_sync(0xffffffffu, ok);
          off[y] = ok ? now.page[y] * a.cache.page_stride + now.place[y] * a.cache.token_stride + now.head * (D * 2) : -1ll;
        }
        now = next;
        look_up();
        if (tile_no < 0) continue;
        if (!is_v && lane == 0) sh.valid[tile_no % kAhead] = make_uint2(exist[0], exist[1]);
        wait(&sh.empty[slot], turn & 1);
        const uint32_t dst = ring + slot * L::kSlot;
        // (rows that do not exist are zero-filled)
        if (in_page) {
#pragma unroll 4
          for (int g = 0; g < 8; ++g) {
            const long long first = __shfl_sync(0xffffffffu, g < 4 ? off[0] : off[1], (g & 3) * 8);  // -1: nor do the rest
            const uint32_t some = (g < 4 ? exist[0] : exist[1]) >> ((g & 3) * 8 + r0);
            const char* from = first < 0 ? a.cache.k : pool + first;
            const long long on = first < 0 ? 0 : stride;
#pragma unroll
            for (int i = 0; i < kPasses; ++i, from += on)
              cp16(dst + (g * 8 + i * kStep) * 128 + (((chunk & 7) ^ ((r0 + i * kStep) & 7)) << 4), from, ((some >> (i * kStep)) & 1) << 4, policy);
          }
        } else {
#pragma unroll 8
          for (int i = 0; i < 8 * kPasses; ++i) {
            const int t = r0 + i * kStep;
            const long long from = __shfl_sync(0xffffffffu, i < 4 * kPasses ? off[0] : off[1], t & 31) - r0 * a.cache.token_stride;
            const bool some = ((i < 4 * kPasses ? exist[0] : exist[1]) >> (t & 31)) & 1;
            cp16(dst + i * kStep * 128 + (((chunk & 7) ^ (t & 7)) << 4), some ? pool + from : a.cache.k, some ? 16 : 0, policy);
          }
        }
        cp_arrive(&sh.full[slot]);
        if (lane == 0) mbar_arrive(&sh.full[slot]);  // (the tokens' bits come with it)
        slot += 4;
        if (slot >= kSlots) {
          slot -= kSlots;
          ++turn;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");  // no copy is under way when the block leaves
    } else if (warp == kScores) {
      // ---- scores ----------------------------------------------------------------
      const uint32_t ring = smem_addr(smem), q_at = smem_addr(q_s);
      int count0 = 0, count1 = 0, tile_no = 0, items = 0;  // tiles of the streams, where they differ; of both
      for (;; ++items) {
        const Item& at = item(items);
        if (!at.any) break;
        const int tiles = at.tile1 - at.tile0;
        for (int j = 0; j < tiles; ++j, ++tile_no) {
          const int slot = (2 * tile_no) % kSlots;
          if (j == 0) wait(&sh.q_full, items & 1);
          wait(&sh.full[slot], ((2 * tile_no) / kSlots) & 1);
          async_fence();  // the copies, to the products
#pragma unroll 1
          for (int s = kDual ? 0 : j & 1; s < (kDual ? 2 : (j & 1) + 1); ++s) {
            const int c = kDual ? tile_no : s ? count1++ : count0++, buf = c & 1;
            wait(&sh.pv_done[s][buf], ((c >> 1) + 1) & 1);  // (the first of a buffer finds it free)
            tc_after();
            scores_mma<D>(tmem + s * kStream + buf * kTile, operand(q_at + (kDual ? s : 0) * (128 * D * 2), 16, 1024, 2),
                          operand(ring + slot * L::kSlot, 16, 1024, 2));
            if (!kDual || s == 1) {
              tc_commit(&sh.empty[slot]);
              if (j == tiles - 1) tc_commit(&sh.q_free);
            }
            tc_commit(&sh.s_full[s][buf]);
          }
        }
      }
      if (*reinterpret_cast<volatile int*>(&sh.dead)) {  // none of them may be under way when TMEM is freed
        tc_commit(&sh.done[0]);
        mbar_wait_sleep(&sh.done[0], 0);
      }
      __syncwarp();
    } else if (warp == kOutputs) {
      // ---- outputs -----------------------------------------------------------------
      const uint32_t ring = smem_addr(smem);
      int count0 = 0, count1 = 0, tile_no = 0;
      for (int items = 0;; ++items) {
        const Item& at = item(items);
        if (!at.any) break;
        const int tiles = at.tile1 - at.tile0;
        for (int j = 0; j < tiles; ++j, ++tile_no) {
          const int slot = (2 * tile_no + 1) % kSlots;
          wait(&sh.full[slot], ((2 * tile_no + 1) / kSlots) & 1);
#pragma unroll 1
          for (int s = kDual ? 0 : j & 1; s < (kDual ? 2 : (j & 1) + 1); ++s) {
            const int c = kDual ? tile_no : s ? count1++ : count0++, buf = c & 1;
            wait(&sh.p_full[s][buf], (c >> 1) & 1);
            async_fence();
            tc_after();
            outputs_mma<D>(tmem + s * kStream + kO, tmem + s * kStream + buf * kTile, operand(ring + slot * L::kSlot, kHalf, 1024, 2),
                           kDual ? j > 0 : j > 1);
            if (!kDual || s == 1) tc_commit(&sh.empty[slot]);
            tc_commit(&sh.pv_done[s][buf]);
          }
        }
      }
      if (*reinterpret_cast<volatile int*>(&sh.dead)) {
        tc_commit(&sh.done[1]);
        mbar_wait_sleep(&sh.done[1], 0);
      }
      __syncwarp();
    } else if (warp == kWalker) {
      // ---- items -------------------------------------------------------------------
      Walker<L::kRows, kEndR<kDual>> at(a, z, lane);
      for (int items = 0;; ++items) {
        Item i;
        at.next(i);
        wait(&sh.item_free[items % kItems], (items / kItems + 1) & 1);  // (the first ones are)
        if (*reinterpret_cast<volatile int*>(&sh.dead)) break;             // (an item that is read stays)
        if (lane == 0) {
          sh.item[items % kItems] = i;
          mbar_arrive(&sh.item_ready[items % kItems]);
        }
        __syncwarp();
        if (!i.any) break;
      }
    } else {
      // ---- queries, from the second item on --------------------------------------------
      for (int items = 0;; ++items) {
        const Item& at = item(items);
        if (!at.any) break;
        if (items == 0) continue;
        wait(&sh.q_free, (items - 1) & 1);  // the scores of the item before are done
#pragma unroll 1
        for (int y = 0; y < L::kRows / 32; ++y) load_q(at, y);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    // ---- softmax: a row a thread --------------------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int s = warp >> 2, row_in = tid & 127, quad = warp & 3;
    const int row_at = kDual ? s * 128 : 0;  // the stream's first row of an item
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_col = tmem + lanes + s * kStream, o_col = s_col + kO;
    const float scale = a.scale_log2;  // above zero
    TreeSight<128>& sight = sh.sight[s];
    if (warp < L::kRows / 32) {  // the first item's queries
      const Item& at = item(0);
      if (at.any) load_q(at, warp);
    }
    int count = 0, tile_no = 0, sight_b = -1, sight_rt = -1;
    for (int items = 0;; ++items) {
      const Item& at = item(items);
      // (those that meet at barriers below stop together, also where a wait ran out)
      if (kDual ? any_of(3 + s, 128, !at.any) : any_of(1, 256, !at.any)) break;
      // Nobody reads the item before the last any more: every warp has read it before it
      // could do what the last one needed of it.  (The last one itself may still be ahead of
      // the queries' warp, where it is the block's first, and of the loaders of odd
      // tiles, where it is that and one tile: the softmax warps needed nothing of theirs.)
      if (items >= kHeld && row_in == 0) mbar_arrive(&sh.item_free[(items - kHeld) % kItems]);
      const int base = at.n - a.Q;
      if (at.b != sight_b || at.rt != sight_rt) {
        stream_sync(s);
        tree_sight<128>(a, at.b, base, at.row0 + row_at, at.row0 + at.rows - 1, row_in, 128, sight, [&] { stream_sync(s); });
        sight_b = at.b;
        sight_rt = at.rt;
      }
      if (tid == 0) sh.odd[(items + kOdd / 2) % kOdd] = 0;
      float m = -INFINITY, l = 0.f;
      const int tile0 = at.tile0, tiles = at.tile1 - tile0;
      const int first = kDual ? 0 : s, step = kDual ? 1 : 2;
      for (int j = first; j < tiles; j += step, ++count) {
        const int buf = count & 1, t0 = (tile0 + j) * kTile, now = tile_no + j;
        wait(&sh.s_full[s][buf], (count >> 1) & 1);
        tc_after();
        const uint32_t at_s = s_col + buf * kTile;
        const uint2 valid = sh.valid[now % kAhead];
        // a tile whose tokens all exist and come before the tree needs no mask
        const bool masked = (valid.x & valid.y) != 0xffffffffu || t0 + kTile > base;
        // A value that is not finite would reach rows that do not see its token as 0 *
        // inf: such values are zero in the products, and added to the rows that see
        // them at the end.  (Tokens that do not exist are zero-filled.  The first
        // stream does it for both: the second's products with the tile are issued
        // after the first's.)
        if (t0 + kTile > base && (!kDual || s == 0)) {
          const int slot = (2 * now + 1) % kSlots, token = row_in & (kTile - 1);
          wait(&sh.full[slot], ((2 * now + 1) / kSlots) & 1);
          if (t0 + token >= base) {
            uint4* v = reinterpret_cast<uint4*>(smem + slot * L::kSlot + token * 128);
            bool odd = false;
#pragma unroll 4
            for (int i = 0; i < kChunks / 2; ++i) {
              const int c = (row_in >> 6) * (kChunks / 2) + i;
              uint4* piece = v + (c >> 3) * (kHalf / 16) + ((c ^ token) & 7);  // (in an order without bank conflicts)
              const uint4 w = *piece;
              if (nonfinite2(w.x) || nonfinite2(w.y) || nonfinite2(w.z) || nonfinite2(w.w)) {
                odd = true;
                *piece = make_uint4(mma::even_word<BF16>(w.x), mma::even_word<BF16>(w.y), mma::even_word<BF16>(w.z), mma::even_word<BF16>(w.w));
              }
            }
            if (odd) {
              sh.odd[items % kOdd] = 1;
              async_fence();
            }
          }
        }
        uint32_t x[64];
        ld64(x, at_s);
        if (masked) {
          const uint32_t see[2] = {valid.x & sight.window(row_in, t0 - base), valid.y & sight.window(row_in, t0 + 32 - base)};
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (!((see[i >> 5] >> (i & 31)) & 1)) x[i] = 0xff800000u;  // -inf
        }
        float top = -INFINITY;
        {
          float y[3] = {-INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 64; i += 8) {
            top = max3(top, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
#pragma unroll
            for (int k = 0; k < 3; ++k) y[k] = max3(y[k], __uint_as_float(x[i + 2 + 2 * k]), __uint_as_float(x[i + 3 + 2 * k]));
          }
          top = fmaxf(max3(top, y[0], y[1]), y[2]);
        }
        top *= scale;
        const bool grow = top > m + kSlackR;
        if (__any_sync(0xffffffffu, grow)) {
          const float c = grow ? (m == -INFINITY ? 0.f : ex2(m - top)) : 1.f;
          if (grow) m = top;
          if (j > first) {
            l *= c;
            wait(&sh.pv_done[s][buf ^ 1], ((count - 1) >> 1) & 1);  // O is complete
            tc_after();
#pragma unroll 1
            for (int d = 0; d < D; d += 16) {
              uint32_t o[16];
              ld16(o, o_col + d);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * c);
              st16(o_col + d, o);
            }
          }
        }
        const float less = m == -INFINITY ? 0.f : -m;
        const uint64_t scale2 = pair(__float_as_uint(scale), __float_as_uint(scale)), less2 = pair(__float_as_uint(less), __float_as_uint(less));
        const uint64_t minus2 = pair(0xbf800000u, 0xbf800000u);  // -1
        uint64_t sum0 = 0, sum1 = 0;                             // (two fp32 zeros)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float p0, p1;
            split(fma2(pair(x[h * 32 + 2 * i], x[h * 32 + 2 * i + 1]), scale2, less2), p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            const uint64_t p = pair(__float_as_uint(p0), __float_as_uint(p1));
            if (i & 1) sum1 = add2(sum1, p);
            else sum0 = add2(sum0, p);
            hi[i] = pack2(p0, p1);
            split(fma2(pair(hi[i] << 16, hi[i] & 0xffff0000u), minus2, p), p0, p1);
            lo[i] = pack2(p0, p1);
          }
          st16(at_s + h * 32, hi);
          st16(at_s + h * 32 + 16, lo);
        }
        {
          float a0, a1;
          split(add2(sum0, sum1), a0, a1);
          l += a0 + a1;
        }
        tmem_st_done();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[s][buf]);
      }

      // ---- the item, or this block's part of it ---------------------------------
      const int r = row_at + row_in;  // of the item
      const bool row = r < at.rows, none = sight.blind(row_in);
      const AttnRow ar = row_of(z, at.row0 + min(r, at.rows - 1), at.h);
      const size_t to = (static_cast<size_t>(at.b) * a.Q + ar.i) * a.Hq + ar.hq;
      float* slot = attn_slot<L::kRows, D>(a, blockIdx.x, at.tile0 == 0);
      const uint32_t rows = __ballot_sync(0xffffffffu, row);
      long long to4[4];  // the four lanes' rows
#pragma unroll
      for (int k = 0; k < 4; ++k) to4[k] = __shfl_sync(0xffffffffu, static_cast<long long>(to), (lane & 28) | k);
      const bool mine = tiles > first;  // has the stream a part
      if (mine) wait(&sh.pv_done[s][(count - 1) & 1], ((count - 1) >> 1) & 1);
      const bool whole = at.whole();
      float c0 = 1.f, c1 = 0.f;  // of the streams' parts
      bool both = false;
      if constexpr (!kDual) {
        sh.m[s][row_in] = m;
        sh.l[s][row_in] = l;
        soft_sync();
        both = tiles > 1;
        const float m0 = sh.m[0][row_in], m1 = sh.m[1][row_in];
        m = fmaxf(m0, m1);
        // (a part without a maximum holds zeros, or NaN that it passes on)
        c0 = m0 == -INFINITY ? 1.f : ex2(m0 - m);
        c1 = m1 == -INFINITY ? 1.f : ex2(m1 - m);
        l = c0 * sh.l[0][row_in];
        if (both) l = fmaf(c1, sh.l[1][row_in], l);
      }
      tc_after();
      if (none) {  // no node: what it summed over the context is nobody's
        m = -INFINITY;
        l = 0.f;
      }
      const float inv = whole ? (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) : 1.f;
      const bool odd = *reinterpret_cast<volatile int*>(&sh.odd[items % kOdd]) != 0;
      constexpr int kPart = kDual ? D : D / 2;  // columns that the thread writes
      c0 *= inv;
      c1 *= inv;
#pragma unroll 1
      for (int d = kDual ? 0 : s * kPart, end = d + kPart; d < end; d += 32) {
        uint32_t u[32];
        float o[32];
        ld32(u, tmem + lanes + (kDual ? s * kStream : 0) + kO + d);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = none ? 0.f : __uint_as_float(u[i]) * c0;
        if (!kDual && both) {
          ld32(u, tmem + lanes + kStream + kO + d);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = none ? 0.f : fmaf(c1, __uint_as_float(u[i]), o[i]);
        }
        if (whole) {
          // A row's 16-byte pieces change places with those of the three rows beside it,
          // so that four lanes write 64 bytes of a row together.
          uint32_t w[4][4];
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i >> 2][i & 3] = pack2(o[2 * i], o[2 * i + 1]);
#pragma unroll
          for (int bit = 1; bit < 4; bit <<= 1)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (!(k & bit))
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const bool up = lane & bit;
                  const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[k][i] : w[k | bit][i], bit);
                  if (up) w[k][i] = got;
                  else w[k | bit][i] = got;
                }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if ((rows >> ((lane & 28) | k)) & 1)
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + to4[k] * D + d + (lane & 3) * 8) =
                  make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
        } else if (row) {
          float4* out = reinterpret_cast<float4*>(slot) + d / 4 * L::kRows + r;  // (parts lie by four dimensions, then rows)
#pragma unroll
          for (int i = 0; i < 8; ++i) out[i * L::kRows] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      __syncwarp();
      if (odd && row && !none) {
        constexpr int kFrom = kDual ? 0 : kPart;
#pragma unroll 1
        for (int t = max(at.tile0 * kTile, max(base, 0)); t < min(at.tile1 * kTile, at.n); ++t) {
          if (!sight.sees(row_in, t - base)) continue;
          const int entry = static_cast<int>(z.by_page(static_cast<unsigned long long>(t)));
          const int page = a.table.ids[at.b * a.table.stride + entry];
          if (page < 0 || page >= a.cache.pages) continue;
          const char* v = a.cache.v + page * a.cache.page_stride + (t - entry * a.cache.page_size) * a.cache.token_stride +
                          at.h * (D * 2);
#pragma unroll 1
          for (int d = s * kFrom; d < s * kFrom + kPart; ++d) {
            const float y = load_one<BF16>(v, d);
            if (isfinite(y)) continue;
            if (whole) {
              uint16_t* out = static_cast<uint16_t*>(a.out) + to * D + d;
              *out = static_cast<uint16_t>(pack2(__uint_as_float(static_cast<uint32_t>(*out) << 16) + y, 0.f));
            } else {
              slot[(d / 4 * L::kRows + r) * 4 + d % 4] += y;
            }
          }
        }
      }
      if (row && (kDual || s == 0)) {
        if (!whole) {
          slot[L::kRows * D + r] = m;
          slot[L::kRows * D + L::kRows + r] = l;
        } else if (a.lse) {
          a.lse[to] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
      }
      tc_before();  // O has been read
      if (!whole && at.tile0 == 0 && tid == 0) joins[blockIdx.x] = {at.b, at.h, at.row0, at.rows, at.end, 0};
      if constexpr (!kDual) soft_sync();  // both streams' O may be written again
      tile_no += tiles;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  if (warp == kOutputs) {
    tc_after();
    if (lane == 0 && sh.dead && a.status) atomicOr(a.status, kWaitTimeout);
    tmem_free(tmem, kCols);
  }
}

// Blocks [block, end] of the launch have left (m, l, O) of a cut item.  A warp joins
// 8 dimensions of 32 rows, a row a lane, in block order, two parts' loads under way
// together.  (Little code: more parts at a time took longer, to fetch it.)
constexpr int kJoinWarps = 4, kJoinDims = 8;
template <int D, bool kDual>
__global__ void __launch_bounds__(kJoinWarps * 32) tree_join_kernel(const AttnArgs a, const Shape z, const Join* joins) {
  constexpr int kRows = Lay<D, kDual>::kRows, kSplit = D / kJoinDims / kJoinWarps;  // blocks that share 32 rows
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Join j = joins[blockIdx.x];
  const int first = blockIdx.x, lane = threadIdx.x & 31;
  const int r0 = blockIdx.y / kSplit * 32, d0 = (blockIdx.y % kSplit * kJoinWarps + (threadIdx.x >> 5)) * kJoinDims;
  if (r0 >= j.rows) return;
  const int r = min(r0 + lane, j.rows - 1);
  float m = -INFINITY, l = 0.f, o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.f;
#pragma unroll 1
  for (int c0 = first; c0 <= j.end; c0 += 2) {
    float mc[2], lc[2];
    float4 v[2][2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int c = min(c0 + y, j.end);
      const float* s = attn_slot<kRows, D>(a, c, c == first);
      mc[y] = s[kRows * D + r];
      lc[y] = s[kRows * D + kRows + r];
#pragma unroll
      for (int i = 0; i < 2; ++i) v[y][i] = *reinterpret_cast<const float4*>(s + ((d0 / 4 + i) * kRows + r) * 4);
    }
    const float before = m;
    m = fmaxf(m, fmaxf(mc[0], mc[1]));
    const float keep = before == -INFINITY ? 1.f : ex2(before - m);
    l *= keep;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= keep;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      if (c0 + y > j.end) break;
      const float w = mc[y] == -INFINITY ? 1.f : ex2(mc[y] - m);  // a part without a maximum holds zeros, or NaN that it passes on
      l = fmaf(w, lc[y], l);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        o[4 * i] = fmaf(w, v[y][i].x, o[4 * i]);
        o[4 * i + 1] = fmaf(w, v[y][i].y, o[4 * i + 1]);
        o[4 * i + 2] = fmaf(w, v[y][i].z, o[4 * i + 2]);
        o[4 * i + 3] = fmaf(w, v[y][i].w, o[4 * i + 3]);
      }
    }
  }
  if (r0 + lane >= j.rows) return;
  const AttnRow ar = row_of(z, j.row0 + r, j.h);
  const size_t at = (static_cast<size_t>(j.b) * a.Q + ar.i) * a.Hq + ar.hq;
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at * D + d0) =
      make_uint4(pack2(o[0] * inv, o[1] * inv), pack2(o[2] * inv, o[3] * inv), pack2(o[4] * inv, o[5] * inv), pack2(o[6] * inv, o[7] * inv));
  if (d0 == 0 && a.lse) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int D, bool kDual>
cudaError_t prepare() {
  return cudaFuncSetAttribute(attention_tree_kernel<D, kDual>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D, kDual>::kBytes);
}
template <int D, bool kDual>
size_t workspace() {
  return static_cast<size_t>(kAttnMaxCtas) * 4 + static_cast<size_t>(kMaxCtas) * (2 * Lay<D, kDual>::kRows * (D + 2) * 4 + sizeof(Join));
}
template <int D, bool kDual>
cudaError_t launch(const AttnArgs& a, int sm_count, cudaStream_t stream) {
  using L = Lay<D, kDual>;
  const int grid = sm_count < kMaxCtas ? sm_count : kMaxCtas;
  Join* joins = reinterpret_cast<Join*>(a.partials + static_cast<size_t>(kMaxCtas) * 2 * L::kRows * (D + 2));
  Shape z;
  z.G = a.Hq / a.cache.heads;
  z.R = a.Q * z.G;
  z.RT = (z.R + L::kRows - 1) / L::kRows;
  z.by_page = DivU64::make(static_cast<unsigned long long>(a.cache.page_size));
  z.by_group = DivU64::make(static_cast<unsigned long long>(z.G));
  z.by_heads = DivU64::make(static_cast<unsigned long long>(a.cache.heads));
  z.by_items = DivU64::make(static_cast<unsigned long long>(a.cache.heads) * z.RT);
  AttnArgs b = a;
  b.whole = static_cast<int64_t>(a.table.max_pages) * a.cache.page_size <= kWholeTiles * kTile &&
            static_cast<int64_t>(a.B) * a.cache.heads * z.RT <= grid;  // by the room of the page tables alone
  attention_tree_kernel<D, kDual><<<grid, kThreadsR, L::kBytes, stream>>>(b, z, joins);
  if (b.whole) return cudaGetLastError();  // nothing to join
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, ((z.R < L::kRows ? z.R : L::kRows) + 31) / 32 * (D / kJoinDims / kJoinWarps));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute after[1];
  after[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  after[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = after;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, tree_join_kernel<D, kDual>, b, z, static_cast<const Join*>(joins));
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace ttc
}  // namespace specv
