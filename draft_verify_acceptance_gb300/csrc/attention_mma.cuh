// attention_mma.cuh -- paged attention on the tensor cores, bf16 and fp32 (sm_103a).
//
// Decode attention reads every cached byte for a handful of rows, so HBM is
// the bound and the tensor cores only have to keep out of its way.  The
// products are taken transposed,
//     S^T [tokens x rows] = K Q^T,   O^T [D x rows] += V^T P^T,
// which puts the long dimensions (tokens, D) on the 16-row side of
// mma.m16n8k16 and the few rows on its 8-column side: 4 rows cost one column
// block and 24 cost three, where rows on the 16-row side would cost two and
// four.  It also leaves a row's running maximum, its sum and its column of
// O^T in the same threads.  P^T changes from accumulator to operand layout
// by one 8 x 8 transpose (movmatrix) per 8 tokens.  A weight enters the second
// product as the sum of two bf16 values (16 significant bits): one bf16 weight
// would lose up to 2^-8 of each term, as much as rounding the output does, and
// the extra product is hidden behind HBM.
//
// Every warp streams tokens of its own: 16 a step through a private ring of
// kStages steps in shared memory (cp.async, 16-byte pieces, XOR-swizzled
// rows), so warps wait for their own loads alone and the block meets only at
// the end of an item.  A row's reference maximum moves only when a score
// passes it by 2^8 (the weights then stay below 2^8, which fp32 sums carry
// without loss), so most steps need no reduction across
// lanes and no rescaling.
//
// Measured, bf16, heads of 128, 32 query heads on 8: one query on 64 sequences
// of 4000 tokens 166 us (the cache's bytes at the copy rate: 157), on 64 of
// 400..4000 101 (94), on 3 of 60001..131072 200 to 215 (190; it differs by
// machine); six queries on the ragged 64 107 to 116 (94): HBM is the bound
// until 24 rows' 72 products a step and an item's end (some 4 us: the ring
// drains, the warps' parts meet) show.
//
// fp32 takes m16n8k8 on tf32 parts: x = hi + lo with hi = x rounded to 11 bits
// and lo the rest, and a product as hi hi + hi lo + lo hi, each exact in fp32,
// which leaves out 2^-22 of a term.  The tensor cores' sums are not rounded to
// nearest, so no chain of them is long: a score's hi parts make two chains of
// D / 16 and the rest a third, and a step's part of O^T starts from zero and
// is added by an fp32 add.  32 sequences of 400..4000 tokens take 141 us for one
// query and 234 for six (97): neither HBM (59 and 36 %) nor the issue slots (40
// and 34 %) nor the tensor cores (20 and 36 %) are full, and a warp waits most
// for results of its own (fixed latencies, then the tensor pipe): six warps an
// SM, which is what the ring leaves room for, are too few to cover them.
#pragma once

#include "attention_common.cuh"
#include "tree_common.cuh"

namespace specv {
namespace mma {

constexpr int kMaxMmaCtas = 304;             // blocks of a launch
constexpr int kMmaRows = 24;                 // rows of an item, at most
constexpr int kTokens = 16;                  // a warp's step
constexpr float kSlack = 8.f;                // how far (log2) a score may pass the reference

template <typename E, int D, int NB, int kTree = 0>
struct Ring {
  static constexpr bool kF32 = E::kBytes == 4;
  static constexpr bool kWide = kTree == 2;  // one block of eight warps an SM
  static_assert(!kWide || (kF32 && D == 64), "the others fill an SM with their rings");
  static constexpr int kWarps = kF32 && D == 128 ? 6 : kWide ? 8 : 4;
  static constexpr int kStages = kF32 ? (D == 128 ? 2 : 3) : (D == 128 ? 3 : 6);
  static constexpr int kCtas = (kF32 && D == 128) || kWide ? 1 : 2;  // an SM holds
  static constexpr int kEnd = kF32 ? NB + 1 : 2 * NB + 2;  // steps that an item's start and end count as
  static constexpr int kRow = D * E::kBytes;             // bytes of a token's K or V
  static constexpr int kHalf = kTokens * kRow;           // K of a step; V follows
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kRing = kWarps * kStages * kStage;
  // fp32 queries, split, as operand fragments: [NB][D / 16][hi, lo][32 lanes][16 bytes]
  static constexpr int kQueries = kF32 ? NB * (D / 16) * 1024 : 0;
  static constexpr int kBytes = kRing + kQueries;
};

// Where 16-byte piece `chunk` of token r's row lies in it, so that the lanes
// that read together meet different banks.
template <typename E>
__device__ __forceinline__ int k_place(int chunk, int r) {
  if constexpr (E::kBytes == 4) return chunk ^ ((r & 1) << 2);
  else return chunk ^ (r & 7);
}
template <typename E>
__device__ __forceinline__ int v_place(int chunk, int r) {
  if constexpr (E::kBytes == 4) return chunk ^ (r & 6);
  else return chunk ^ (r & 7);
}
// Dimension of half y (of 8) of lane group g's rows of tile mt of O^T.  fp32
// lanes read four dimensions at once, which go to four tiles.
template <typename E>
__device__ __forceinline__ int dim_of(int mt, int y, int g) {
  if constexpr (E::kBytes == 4) return (mt >> 2) * 64 + y * 32 + g * 4 + (mt & 3);
  else return mt * 16 + y * 8 + g;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma1688(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x as two tf32 parts; what is not finite, or rounds to infinity (from
// kTf32Inf on), is whole in the first.
constexpr uint32_t kTf32Inf = 0x7f7ff000u;
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
  lo = (hi & 0x7f800000u) == 0x7f800000u ? 0u : __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ float4 lds4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}
template <typename E>
__device__ __forceinline__ float shared_value(uint32_t at) {
  if constexpr (E::kBytes == 4) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
  } else {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
  }
}
__device__ __forceinline__ uint4 lds4u(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ bool nonfinite2(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
// Is a word of the cache, one fp32 or two bf16 values, not all finite as an
// operand; and it with zero in place of what is not.
template <typename E>
__device__ __forceinline__ bool odd_word(uint32_t w) {
  return E::kBytes == 4 ? (w & 0x7fffffffu) >= kTf32Inf : nonfinite2(w);
}
template <typename E>
__device__ __forceinline__ uint32_t even_word(uint32_t w) {
  if (E::kBytes == 4) return odd_word<E>(w) ? 0u : w;
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
  return w;
}

// NB blocks of 8 rows an item.  kTree 1 and 2: the queries are a tree's nodes, and see
// its tokens by TreeSight's bits instead of up to themselves.
template <typename E, int D, int NB, int kTree>
__global__ void __launch_bounds__(Ring<E, D, NB, kTree>::kWarps * 32, Ring<E, D, NB, kTree>::kCtas) attention_mma_kernel(const AttnArgs a, DivU64 by_page) {
  using L = Ring<E, D, NB, kTree>;
  constexpr bool kF32 = L::kF32;
  constexpr int kWarpsM = L::kWarps, kThreadsM = kWarpsM * 32, kStepM = kWarpsM * kTokens;  // a block's step
  constexpr int kRows = 8 * NB, KS = D / 16, kStages = L::kStages;
  constexpr int kRow = L::kRow, kHalf = L::kHalf, kStage = L::kStage;
  constexpr int kChunks = kRow / 16;           // 16-byte pieces of a row
  constexpr int kRowsPer = 32 / kChunks;       // rows a warp's copy instruction covers
  constexpr int kPitch = D + 4;                // of the warps' O in shared memory, floats
  static_assert(kWarpsM * kRows * kPitch * 4 <= L::kRing, "the warps' parts fit the ring");
  extern __shared__ __align__(128) char ring[];
  __shared__ uint32_t s_valid[kWarpsM][kStages];  // which tokens of a step exist
  __shared__ float s_m[kWarpsM][kRows], s_l[kWarpsM][kRows];
  __shared__ long long s_plan[2 * kWarpsM + 4];
  __shared__ int s_flag;
  __shared__ TreeSight<kTree ? kRows : 0> s_tree;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int H = a.cache.heads, G = a.Hq / H, R = a.Q * G;
  const int RT = (R + kRows - 1) / kRows;
  const int S = a.cache.page_size;
  const bool page_steps = S % kTokens == 0;    // a step lies in one page
  char* mine = ring + warp * (kStages * kStage);
  const uint32_t mine_at = smem_addr(mine);

  constexpr int kEnd = L::kEnd;
  AttnPlan plan;
  if (kTree && a.whole) plan = attn_plan_whole<kEnd>(a, H * RT);
  else plan = attn_plan<kStepM, kEnd, kThreadsM>(a, H * RT, 4, s_plan);
  AttnWalk<kStepM, kEnd, kRows> at(a, plan);
  while (at.next()) {
    const int n = at.n, b = at.b, h = at.h, row0 = at.row0, rows = at.rows, tile0 = at.tile0, tile1 = at.tile1;
    const int32_t* table = a.table.ids + b * a.table.stride;

    // The warp's steps: tokens [kStepM * tile + 16 * warp, + 16) of each tile.
    const int first = tile0 * kStepM + warp * kTokens;
    const int last = min(tile1 * kStepM, n);   // tokens of this part end here
    const int steps = first < last ? (last - first + kStepM - 1) / kStepM : 0;

    // Lane l looks up the page of the step's token l % 16.
    auto page_of = [&](int j) -> int {
      const int t = first + j * kStepM + (lane & (kTokens - 1));
      return t < last ? table[static_cast<int>(by_page(static_cast<unsigned long long>(t)))] : 0;
    };
    auto issue = [&](int j, int page) {
      const int t0 = first + j * kStepM;
      const int t = t0 + (lane & (kTokens - 1));
      const bool known = page >= 0 && page < a.cache.pages;
      const bool ok = t < last && known;
      if (t < last && !known && a.status) atomicOr(a.status, kDataPageRange);
      const uint32_t valid = __ballot_sync(0xffffffffu, ok) & 0xffffu;
      const int stage = j % kStages;
      if (lane == 0) s_valid[warp][stage] = valid;
      const int slot = static_cast<int>(by_page(static_cast<unsigned long long>(t)));
      const long long off = (ok ? page * a.cache.page_stride + (t - slot * S) * a.cache.token_stride : 0ll) +
                            h * kRow;
      const int chunk = lane % kChunks, r0 = lane / kChunks;
      const uint32_t dst = mine_at + stage * kStage;
      const char* kp = a.cache.k + chunk * 16;
      const char* vp = a.cache.v + chunk * 16;
      if (page_steps && valid == 0xffffu) {
        const long long o0 = __shfl_sync(0xffffffffu, off, 0) + r0 * a.cache.token_stride;
        kp += o0;
        vp += o0;
#pragma unroll
        for (int i = 0; i < kTokens / kRowsPer; ++i) {
          const int r = r0 + i * kRowsPer;
          const uint32_t d = dst + r * kRow;
          cp16(d + (k_place<E>(chunk, r) << 4), kp, 16);
          cp16(d + kHalf + (v_place<E>(chunk, r) << 4), vp, 16);
          kp += kRowsPer * a.cache.token_stride;
          vp += kRowsPer * a.cache.token_stride;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kTokens / kRowsPer; ++i) {
          const int r = r0 + i * kRowsPer;
          const long long o = __shfl_sync(0xffffffffu, off, r);
          const uint32_t bytes = (valid >> r) & 1 ? 16 : 0;  // 0: the piece is zero-filled
          const uint32_t d = dst + r * kRow;
          cp16(d + (k_place<E>(chunk, r) << 4), kp + o, bytes);
          cp16(d + kHalf + (v_place<E>(chunk, r) << 4), vp + o, bytes);
        }
      }
    };

    __syncthreads();  // the ring is free again
    int page = page_of(0);
#pragma unroll
    for (int j = 0; j < kStages - 1; ++j) {
      const int next = page_of(j + 1);
      if (j < steps) issue(j, page);
      cp_commit();
      page = next;
    }
    if constexpr (kTree) tree_sight<kRows>(a, b, n - a.Q, row0, row0 + rows - 1, tid, kThreadsM, s_tree, [] { __syncthreads(); });

    // Queries as operand fragments (rows past the last are zero), and the
    // last token that each of the thread's rows sees.
    uint32_t qf[NB][kF32 ? 1 : KS][2];
    const uint32_t q_at = smem_addr(ring) + L::kRing + lane * 16;
    if constexpr (kF32) {
      for (int e = tid; e < NB * KS * 32; e += kThreadsM) {
        const int l = e & 31, ks = (e >> 5) % KS, r = (e >> 5) / KS * 8 + (l >> 2);
        const AttnRow ar = attn_row(a, row0 + min(r, rows - 1), h);
        const float4 q = __ldg(reinterpret_cast<const float4*>(
            a.q + b * a.q_batch + ar.i * a.q_token + ar.hq * a.q_head + ks * 64 + (l & 3) * 16));
        uint4 hi, lo;
        split(q.x, hi.x, lo.x);
        split(q.y, hi.y, lo.y);
        split(q.z, hi.z, lo.z);
        split(q.w, hi.w, lo.w);
        if (r >= rows) hi = lo = make_uint4(0, 0, 0, 0);
        uint4* to = reinterpret_cast<uint4*>(ring + L::kRing) + (e >> 5) * 64 + l;
        to[0] = hi;
        to[32] = lo;
      }
      __syncthreads();
    }
    int limit[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = nb * 8 + g;
      const AttnRow ar = attn_row(a, row0 + min(r, rows - 1), h);
      const char* qp = a.q + b * a.q_batch + ar.i * a.q_token + ar.hq * a.q_head + t4 * 4;
      if constexpr (!kF32) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qf[nb][ks][0] = r < rows ? __ldg(reinterpret_cast<const uint32_t*>(qp + ks * 32)) : 0u;
          qf[nb][ks][1] = r < rows ? __ldg(reinterpret_cast<const uint32_t*>(qp + ks * 32 + 16)) : 0u;
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) limit[nb][x] = kTree ? n - a.Q : n - a.Q + (row0 + nb * 8 + t4 * 2 + x) / G;
    }
    // Does the thread's row x of block nb see token t (which exists)?
    auto sees_token = [&](int nb, int x, int t) {
      if constexpr (kTree) return t < limit[nb][x] || s_tree.sees(nb * 8 + t4 * 2 + x, t - limit[nb][x]);
      else return t <= limit[nb][x];
    };

    float o[KS][NB][4], m[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      m[nb][0] = m[nb][1] = -INFINITY;
      l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
      for (int mt = 0; mt < KS; ++mt)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[mt][nb][x] = 0.f;
    }

    for (int j = 0; j < steps; ++j) {
      const int next = page_of(j + kStages);
      cp_wait<kStages - 2>();
      __syncwarp();  // this step has landed, and every lane is done with the one before
      if (j + kStages - 1 < steps) issue(j + kStages - 1, page);
      cp_commit();
      page = next;
      const int t0 = first + j * kStepM;
      const int stage = j % kStages;
      const uint32_t kat = mine_at + stage * kStage, vat = kat + kHalf;
      const uint32_t valid = s_valid[warp][stage];

      // S^T = K Q^T
      float s[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[nb][x] = 0.f;
      if constexpr (kF32) {
        float more[NB][4], rest[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int x = 0; x < 4; ++x) more[nb][x] = rest[nb][x] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const float4 k0 = lds4(kat + g * kRow + (k_place<E>(ks * 4 + t4, g) << 4));
          const float4 k8 = lds4(kat + (g + 8) * kRow + (k_place<E>(ks * 4 + t4, g) << 4));
          uint32_t hi[2][4], lo[2][4];
          split(k0.x, hi[0][0], lo[0][0]);
          split(k8.x, hi[0][1], lo[0][1]);
          split(k0.y, hi[0][2], lo[0][2]);
          split(k8.y, hi[0][3], lo[0][3]);
          split(k0.z, hi[1][0], lo[1][0]);
          split(k8.z, hi[1][1], lo[1][1]);
          split(k0.w, hi[1][2], lo[1][2]);
          split(k8.w, hi[1][3], lo[1][3]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const uint4 qh = lds4u(q_at + (nb * KS + ks) * 1024), ql = lds4u(q_at + (nb * KS + ks) * 1024 + 512);
            mma1688(s[nb], hi[0], qh.x, qh.y);
            mma1688(rest[nb], lo[0], qh.x, qh.y);
            mma1688(rest[nb], hi[0], ql.x, ql.y);
            mma1688(more[nb], hi[1], qh.z, qh.w);
            mma1688(rest[nb], lo[1], qh.z, qh.w);
            mma1688(rest[nb], hi[1], ql.z, ql.w);
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[nb][x] = (s[nb][x] + more[nb][x]) + rest[nb][x];
      } else {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const int r = lane & 15, c = ks * 2 + (lane >> 4);
          uint32_t kf[4];
          ldsm4(kf, kat + r * kRow + (k_place<E>(c, r) << 4));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma16816(s[nb], kf, qf[nb][ks][0], qf[nb][ks][1]);
        }
      }
      // a step whose 16 tokens exist and are seen by every row needs no mask
      const bool masked = valid != 0xffffu || t0 + kTokens - 1 > n - a.Q - (kTree ? 1 : 0);
      bool grow = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          s[nb][x] *= a.scale_log2;
          if (masked) {
            const int r = g + (x >> 1) * 8;
            if (!((valid >> r) & 1) || !sees_token(nb, x & 1, t0 + r)) s[nb][x] = -INFINITY;
          }
          grow |= s[nb][x] > m[nb][x & 1] + kSlack;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float mx = fmaxf(s[nb][x], s[nb][x + 2]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            if (!(mx > m[nb][x] + kSlack)) mx = m[nb][x];  // (this row's own scores decide)
            const float c = m[nb][x] == -INFINITY ? 0.f : ex2(m[nb][x] - mx);
            m[nb][x] = mx;
            l[nb][x] *= c;
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
              o[mt][nb][x] *= c;
              o[mt][nb][x + 2] *= c;
            }
          }
      }
      // weights, their sums, and P^T as operand fragments
      uint32_t pf[NB][kF32 ? 8 : 4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float ref = m[nb][x & 1] == -INFINITY ? 0.f : m[nb][x & 1];
          s[nb][x] = ex2(s[nb][x] - ref);
          l[nb][x & 1] += s[nb][x];
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if constexpr (kF32) {
            // the transpose moves 16-bit halves: the lower ones, then the upper
            const uint32_t p0 = __float_as_uint(s[nb][y * 2]), p1 = __float_as_uint(s[nb][y * 2 + 1]);
            const uint32_t low = transpose8(__byte_perm(p0, p1, 0x5410)), up = transpose8(__byte_perm(p0, p1, 0x7632));
            split(__uint_as_float(__byte_perm(low, up, 0x5410)), pf[nb][y * 4], pf[nb][y * 4 + 2]);
            split(__uint_as_float(__byte_perm(low, up, 0x7632)), pf[nb][y * 4 + 1], pf[nb][y * 4 + 3]);
            continue;
          }
          const uint32_t hi = pack2(s[nb][y * 2], s[nb][y * 2 + 1]);
          const uint32_t lo = pack2(s[nb][y * 2] - bf16_lo(hi), s[nb][y * 2 + 1] - bf16_hi(hi));
          pf[nb][y] = transpose8(hi);
          pf[nb][y + 2] = transpose8(lo);
        }
      }
      if (masked) {
        // A value that is not finite would reach rows that do not see its
        // token as 0 * inf.  Such values are added to the rows that do see
        // them one by one, and are zero in the product.
        bool odd = false;
        for (int e = lane; e < kTokens * kChunks; e += 32) {
          const uint4 x = lds4u(vat + e * 16);
          odd |= odd_word<E>(x.x) || odd_word<E>(x.y) || odd_word<E>(x.z) || odd_word<E>(x.w);
        }
        if (__any_sync(0xffffffffu, odd)) {
          for (int t = 0; t < kTokens; ++t) {
            const int from = (t & 7) * 4 + t4;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              float p[2];
              bool sees[2];  // a weight of 0 says nothing: it may have underflowed
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const float lo = __shfl_sync(0xffffffffu, s[nb][x], from);
                const float hi = __shfl_sync(0xffffffffu, s[nb][x + 2], from);
                p[x] = t < 8 ? lo : hi;
                sees[x] = sees_token(nb, x, t0 + t);
              }
#pragma unroll
              for (int mt = 0; mt < KS; ++mt)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const int d = dim_of<E>(mt, y, g), chunk = d * E::kBytes / 16;
                  const float v = shared_value<E>(vat + t * kRow + v_place<E>(chunk, t) * 16 + d * E::kBytes % 16);
                  if (odd_word<E>(__float_as_uint(v))) {
                    if (sees[0]) o[mt][nb][y * 2] += p[0] * v;
                    if (sees[1]) o[mt][nb][y * 2 + 1] += p[1] * v;
                  }
                }
            }
          }
          __syncwarp();
          for (int e = lane; e < kHalf / 4; e += 32) {
            uint32_t* x = reinterpret_cast<uint32_t*>(mine + stage * kStage + kHalf) + e;
            *x = even_word<E>(*x);
          }
          __syncwarp();
        }
      }
      // O^T += V^T P^T
      if constexpr (kF32) {
#pragma unroll
        for (int dg = 0; dg < D / 64; ++dg) {
          float part[4][NB][4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int x = 0; x < 4; ++x) part[i][nb][x] = 0.f;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int r = y * 8 + t4 * 2, c = dg * 16 + g;
            const uint32_t at = vat + r * kRow;
            const float4 v[4] = {lds4(at + (v_place<E>(c, r) << 4)), lds4(at + (v_place<E>(c + 8, r) << 4)),
                                 lds4(at + kRow + (v_place<E>(c, r + 1) << 4)),
                                 lds4(at + kRow + (v_place<E>(c + 8, r + 1) << 4))};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) split(i == 0 ? v[x].x : i == 1 ? v[x].y : i == 2 ? v[x].z : v[x].w, hi[x], lo[x]);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                mma1688(part[i][nb], lo, pf[nb][y * 4], pf[nb][y * 4 + 1]);
                mma1688(part[i][nb], hi, pf[nb][y * 4 + 2], pf[nb][y * 4 + 3]);
                mma1688(part[i][nb], hi, pf[nb][y * 4], pf[nb][y * 4 + 1]);
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int x = 0; x < 4; ++x) o[dg * 4 + i][nb][x] += part[i][nb][x];
        }
      } else {
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
          const int r = (lane & 7) + ((lane >> 4) << 3), c = mt * 2 + ((lane >> 3) & 1);
          uint32_t vf[4];
          ldsm4t(vf, vat + r * kRow + (v_place<E>(c, r) << 4));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma16816(o[mt][nb], vf, pf[nb][0], pf[nb][1]);
            mma16816(o[mt][nb], vf, pf[nb][2], pf[nb][3]);
          }
        }
      }
    }
    cp_wait<0>();

    // ---- the warps' parts, then the item's ----
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[nb][x] += __shfl_xor_sync(0xffffffffu, l[nb][x], 4);
        l[nb][x] += __shfl_xor_sync(0xffffffffu, l[nb][x], 8);
        l[nb][x] += __shfl_xor_sync(0xffffffffu, l[nb][x], 16);
        if (g == 0) {
          s_m[warp][nb * 8 + t4 * 2 + x] = m[nb][x];
          s_l[warp][nb * 8 + t4 * 2 + x] = l[nb][x];
        }
      }
    __syncthreads();  // every warp has left its ring
    float* parts = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int mt = 0; mt < KS; ++mt)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          parts[(warp * kRows + nb * 8 + t4 * 2 + (x & 1)) * kPitch + dim_of<E>(mt, x >> 1, g)] = o[mt][nb][x];
    __syncthreads();
    const bool whole = at.whole();
    float* slot = attn_slot<kRows, D>(a, blockIdx.x, tile0 == 0);
    for (int e = tid; e < rows * (D / 4); e += kThreadsM) {
      const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
      float mm = -INFINITY, ll = 0.f;
      float4 oo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < kWarpsM; ++x) mm = fmaxf(mm, s_m[x][r]);
#pragma unroll
      for (int x = 0; x < kWarpsM; ++x) {
        const float c = s_m[x][r] == -INFINITY ? 0.f : ex2(s_m[x][r] - mm);
        const float4 v = *reinterpret_cast<const float4*>(parts + (x * kRows + r) * kPitch + d);
        ll = fmaf(c, s_l[x][r], ll);
        oo.x = fmaf(c, v.x, oo.x);
        oo.y = fmaf(c, v.y, oo.y);
        oo.z = fmaf(c, v.z, oo.z);
        oo.w = fmaf(c, v.w, oo.w);
      }
      if constexpr (kTree) {
        if (s_tree.blind(r)) {  // no node: what it summed over the context is nobody's
          mm = -INFINITY;
          ll = 0.f;
          oo = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      if (whole) {
        attn_write<D>(a, b, h, row0 + r, d, mm, ll, oo);
      } else {
        *reinterpret_cast<float4*>(slot + r * D + d) = oo;
        if (d == 0) {
          slot[kRows * D + r] = mm;
          slot[kRows * D + kRows + r] = ll;
        }
      }
    }
    if (!whole) {
      if (attn_arrive(a, at.first(), at.tiles, at.per, &s_flag))
        attn_join<kRows, D, kThreadsM>(a, b, h, row0, rows, at.first(), at.tiles, at.per);
    }
  }
}

template <typename E, int D, int NB, int kTree>
cudaError_t prepare() {
  return cudaFuncSetAttribute(attention_mma_kernel<E, D, NB, kTree>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Ring<E, D, NB, kTree>::kBytes);
}
template <typename E, int D, int NB, int kTree>
void launch(const AttnArgs& a, int sm_count, cudaStream_t stream) {
  using L = Ring<E, D, NB, kTree>;
  const int grid = sm_count * L::kCtas < kMaxMmaCtas ? sm_count * L::kCtas : kMaxMmaCtas;
  attention_mma_kernel<E, D, NB, kTree><<<grid, L::kWarps * 32, L::kBytes, stream>>>(
      a, DivU64::make(static_cast<unsigned long long>(a.cache.page_size)));
}
template <typename E, int kTree = 0>
cudaError_t prepare_all() {
  cudaError_t e[] = {prepare<E, 64, 1, kTree>(),  prepare<E, 64, 2, kTree>(),  prepare<E, 64, 3, kTree>(),
                     prepare<E, 128, 1, kTree>(), prepare<E, 128, 2, kTree>(), prepare<E, 128, 3, kTree>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}
// fp32 heads of 64 in blocks of eight warps.
inline void launch_wide(const AttnArgs& a, int nb, int sm_count, cudaStream_t stream) {
  if (nb == 1) launch<F32, 64, 1, 2>(a, sm_count, stream);
  else if (nb == 2) launch<F32, 64, 2, 2>(a, sm_count, stream);
  else launch<F32, 64, 3, 2>(a, sm_count, stream);
}
inline cudaError_t prepare_wide() {
  cudaError_t e[] = {prepare<F32, 64, 1, 2>(), prepare<F32, 64, 2, 2>(), prepare<F32, 64, 3, 2>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}
// Is no item of nb blocks of rows cut, by the room of the page tables alone (attn_plan's rule).
template <typename E, int D, int kTree>
bool whole(const AttnArgs& a, int nb, int sm_count) {
  using L = Ring<E, D, 1, kTree>;  // (the same for all nb in what counts here)
  const int grid = sm_count * L::kCtas < kMaxMmaCtas ? sm_count * L::kCtas : kMaxMmaCtas;
  const int R = a.Q * (a.Hq / a.cache.heads), RT = (R + 8 * nb - 1) / (8 * nb);
  return static_cast<int64_t>(a.table.max_pages) * a.cache.page_size <= kWholeTiles * L::kWarps * kTokens &&
         static_cast<int64_t>(a.B) * a.cache.heads * RT <= grid;
}
// Items of nb blocks of 8 rows, 1 to 3.
template <typename E, int kTree = 0>
void launch_rows(const AttnArgs& a, int nb, int sm_count, cudaStream_t stream) {
  switch (nb + (a.cache.head_dim == 128 ? 3 : 0)) {
    case 1: launch<E, 64, 1, kTree>(a, sm_count, stream); break;
    case 2: launch<E, 64, 2, kTree>(a, sm_count, stream); break;
    case 3: launch<E, 64, 3, kTree>(a, sm_count, stream); break;
    case 4: launch<E, 128, 1, kTree>(a, sm_count, stream); break;
    case 5: launch<E, 128, 2, kTree>(a, sm_count, stream); break;
    default: launch<E, 128, 3, kTree>(a, sm_count, stream); break;
  }
}

}  // namespace mma
}  // namespace specv
