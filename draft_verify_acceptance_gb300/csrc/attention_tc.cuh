// attention_tc.cuh -- bf16 paged attention for more than a few rows a cache
// head (several queries, or many query heads to a cache head), on tcgen05
// (sm_103a).
//
// The products are transposed, as in attention_mma.cuh: tokens and D are the
// long sides, the rows few.
//     S^T [128 tokens x N rows] = K Q^T       A = K tile,   B = Q
//     O^T [D x N rows]         += V^T P^T     A = V^T tile, B = P^T
// Both accumulators live in TMEM (S^T twice, so that the next tile's product
// runs under this tile's softmax), K and V tiles are read from shared memory
// as they come from the cache -- V^T is V's tile read with the other side
// major -- and a tile costs the tensor cores 4 x N x 128 x D multiply-adds
// (P^T counts twice, below), a few hundred cycles where its 64 KB take HBM
// three thousand.
//
// One block per SM.  Warps 8-10 stream tiles through a ring of slots in
// shared memory, K and V in turn, across item boundaries: cp.async in 16-byte
// pieces, whose landing arrives on the slot's barrier by itself, so any page
// size and any strides.  (TMA boxes of a page's tokens, 128 bytes a row, moved
// 23 bytes a cycle an SM however many warps issued them, about what HBM
// delivers and no more.)  Warp 11 issues the products.  Warps 0-3 hold one
// token a thread and half of the rows, warps 4-7 the same tokens and the other
// half: they read S^T, keep each row's reference maximum (moved only when a
// score passes it by 2^8), write the weights P^T as two bf16 parts (hi and
// lo: one bf16 weight would lose up to 2^-8 of a term, as much as rounding the
// output does) and finish items.
//
// 64 sequences of 400..4000 tokens, 8 cache heads of 128: 32 rows a head 168
// us, 68 rows 257 (the cache's bytes at the copy rate: 95).  A tile's softmax
// of 32 rows takes as long as its bytes take HBM, about 2500 cycles (TMEM
// reads, exponentials, the two-part weights' stores), more with more rows; an
// item's start and end, where the ring waits, some 10 us.  Its warps wait for
// TMEM and shared memory and for instructions (each of the roles has code of
// its own); the tensor cores are busy 8 and 14 % of the time.
#pragma once

#include "attention_common.cuh"
#include "attention_mma.cuh"

namespace specv {
namespace tc {

using mma::cp16;
using mma::nonfinite2;
using mma::pack2;

constexpr int D = 128;                   // of a head
constexpr int kTile = 128;               // tokens
constexpr int kSoft = 256;               // softmax threads: two groups of four warps
constexpr int kLoad = 96;                // loader threads
constexpr int kThreadsT = kSoft + kLoad + 32;
constexpr float kSlackT = 8.f;

template <int N>
struct Lay {
  static constexpr int kSlot = kTile * D * 2;   // K or V of a tile
  static constexpr int kQ = N * D * 2;
  static constexpr int kP = kTile * N * 2;      // one part of P^T
  static constexpr int kFree = 216 * 1024 - kQ - 2 * kP;  // (about 9 KB more are static)
  static constexpr int kSlots = kFree / kSlot;
  static constexpr int kBytes = kSlots * kSlot + kQ + 2 * kP + 1024;  // 1024: alignment
  static constexpr int kCols = 3 * N <= 64 ? 64 : 3 * N <= 128 ? 128 : 3 * N <= 256 ? 256 : 512;
  static_assert(kSlots >= 4, "two tiles");
};

// ---- tcgen05 ---------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t* at, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(at)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// The whole warp runs up to these and one lane issues: control flow that the
// warp shares keeps addresses and descriptors in uniform registers (issued
// under `if (lane == 0)` a product took 78 cycles).
// Arrives on `bar` when every product issued so far is done.
__device__ __forceinline__ void tc_commit(unsigned long long* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(float (&v)[8], uint32_t at) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t at, const float (&v)[8]) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_done() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Arrives on `bar` when the thread's copies so far have landed.
__device__ __forceinline__ void cp_arrive(unsigned long long* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory operand: start, leading and stride byte offsets; swizzle 128
// bytes (layout 2) or none (0).
__device__ __forceinline__ uint64_t operand(uint32_t at, uint32_t lead, uint32_t stride, uint32_t layout) {
  return (static_cast<uint64_t>((at & 0x3ffffu) >> 4)) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(stride >> 4) << 32) | (1ull << 46) | (static_cast<uint64_t>(layout) << 61);
}
// bf16 operands, fp32 accumulator, M = 128; `a_mn` / `b_mn`: that operand has
// its M or N side contiguous instead of K.
template <int N>
__device__ __forceinline__ constexpr uint32_t instruction(bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ void load_sync() { asm volatile("bar.sync 2, 96;" ::: "memory"); }
// Group barriers (3 and 4), the second with a vote.
__device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, 128;" ::"r"(3 + group) : "memory"); }
__device__ __forceinline__ bool group_any(int group, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "r"(3 + group)
      : "memory");
  return r != 0;
}

constexpr int kEndT = 6;                 // steps that an item's start and end count as
template <int N>
using Walk = AttnWalk<kTile, kEndT, N>;

template <int N>
struct SharedT {
  unsigned long long full[Lay<N>::kSlots], empty[Lay<N>::kSlots];
  unsigned long long s_full[2], s_free[2], p_full, p_free, q_full, done;
  long long off[2][kTile];             // byte offsets of a tile's tokens, -1: none
  uint32_t valid[8][4];                // tokens that exist, by tile
  float m[N], corr[N], wmax[4][N], lsum[4][N];
  int limit[N];                        // last token that a row sees
  long long q_off[N];                  // of the next item's rows, bytes
  long long out_at[N];                 // of the item's rows: index of [b][i][hq]
  float inv[N];
  int odd;                             // the item has values that are not finite and not every row sees
  uint32_t tmem;
  int dead;                            // a wait ran out: nothing waits any more
  int last;
  long long plan[2 * (kThreadsT / 32) + 4];
};

template <int N>
__global__ void __launch_bounds__(kThreadsT, 1) attention_tc_kernel(const AttnArgs a, DivU64 by_page) {
  using L = Lay<N>;
  constexpr int kSlots = L::kSlots, kHalf = kTile * 128;
  constexpr int kChunks = D / 8;  // 16-byte pieces of a token
  extern __shared__ char raw_smem[];
  __shared__ SharedT<N> sh;
  char* smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  char* q_s = smem + kSlots * L::kSlot;  // [halves][N][128 bytes]
  char* p_s = q_s + L::kQ;               // [hi, lo][N / 8][128 tokens][16 bytes]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  auto wait = [&](unsigned long long* bar, uint32_t parity) {
    if (*reinterpret_cast<volatile int*>(&sh.dead)) return;
    bool gave_up = false;
#ifdef SPEC_DEBUG
    // (a test's way to a wait that ran out: a bit of the status word that it passes)
    gave_up = blockIdx.x == 0 && a.status && (*reinterpret_cast<volatile int32_t*>(a.status) >> 30) != 0;
#endif
    if (gave_up || !mbar_wait_sleep(bar, parity)) {
      *reinterpret_cast<volatile int*>(&sh.dead) = 1;
      if (a.status) atomicOr(a.status, kWaitTimeout);
    }
  };

  const AttnPlan plan = attn_plan<kTile, kEndT, kThreadsT>(
      a, a.cache.heads * ((a.Q * (a.Hq / a.cache.heads) + N - 1) / N), 2, sh.plan);
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sh.full[i], kLoad);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_free[i], kSoft);
    }
    mbar_init(&sh.p_full, kSoft);
    mbar_init(&sh.p_free, 1);
    mbar_init(&sh.q_full, kSoft);
    mbar_init(&sh.done, 1);
    sh.dead = 0;
    fence_barrier_init();
  }
  if (warp == 11) tmem_alloc(&sh.tmem, L::kCols);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = sh.tmem;
  Walk<N> at(a, plan);

  if (warp >= 8 && warp < 11) {
    // ---- K and V of each tile, in turn -----------------------------------
    const int lt = tid - kSoft, S = a.cache.page_size;
    const int chunk = lt % kChunks, r0 = lt / kChunks;
    constexpr int kStep = kLoad / kChunks, kRows = (kTile + kStep - 1) / kStep, kLook = (kTile + kLoad - 1) / kLoad;
    // The tile whose pages are looked up, one ahead of the copies: the table's
    // entries are on their way while the tile before is copied.
    Walk<N> ahead(a, plan);
    bool more = ahead.next();
    int ahead_tile = more ? ahead.tile0 : 0;
    int page[kLook], place[kLook], head = 0;  // place: token in the page, -1: past the end
    auto look_up = [&]() {
      head = ahead.h;
#pragma unroll
      for (int i = 0; i < kLook; ++i) {
        const int t = ahead_tile * kTile + i * kLoad + lt;
        const bool in = t < ahead.n && i * kLoad + lt < kTile;
        const int entry = static_cast<int>(by_page(static_cast<unsigned long long>(t)));
        place[i] = in ? t - entry * S : -1;
        page[i] = in ? __ldg(a.table.ids + ahead.b * a.table.stride + entry) : -1;
      }
      if (++ahead_tile == ahead.tile1) {
        more = ahead.next();
        if (more) ahead_tile = ahead.tile0;
      }
    };
    const bool any = more;
    if (any) look_up();
    // where the thread's piece of row r0 + i * kStep lies in the swizzled slot:
    // the rows' low three bits go round every four steps
    uint32_t place_of[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      place_of[i] = (chunk >> 3) * kHalf + r0 * 128 + (((chunk & 7) ^ ((r0 + i * kStep) & 7)) << 4);
    static_assert(4 * kStep % 8 == 0, "four steps go round");
    int slot = 0;
    uint32_t turn = 0;  // times the ring went round
    for (int tile_no = 0; any; ++tile_no) {
      bool all = true;
#pragma unroll
      for (int i = 0; i < kLook; ++i) {
        const bool ok = page[i] >= 0 && page[i] < a.cache.pages;
        if (!ok && place[i] >= 0 && a.status) atomicOr(a.status, kDataPageRange);
        const uint32_t valid = __ballot_sync(0xffffffffu, ok);
        const int word = i * (kLoad / 32) + warp - kSoft / 32;
        if (word < 4) {
          if (lane == 0) sh.valid[tile_no & 7][word] = valid;
          sh.off[tile_no & 1][i * kLoad + lt] =
              ok ? page[i] * a.cache.page_stride + place[i] * a.cache.token_stride + head * (D * 2) : -1ll;
        }
      }
      load_sync();
      const bool last = !more;
      if (more) look_up();
      const uint32_t* valid = sh.valid[tile_no & 7];
      all = (valid[0] & valid[1] & valid[2] & valid[3]) == 0xffffffffu;
      const long long* off = sh.off[tile_no & 1] + r0;
#pragma unroll 1
      for (int x = 0; x < 2; ++x) {
        if (turn > 0) wait(&sh.empty[slot], (turn + 1) & 1);
        const char* pool = (x ? a.cache.v : a.cache.k) + chunk * 16;
        const uint32_t dst = smem_addr(smem) + slot * L::kSlot;
        if (lt < kStep * kChunks) {
          // (offsets are read ahead of the copies, which no load passes)
#pragma unroll
          for (int i0 = 0; i0 < kRows; i0 += 8) {
            long long from[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i0 + i < kRows && ((i0 + i + 1) * kStep <= kTile || r0 + (i0 + i) * kStep < kTile))
                from[i] = off[(i0 + i) * kStep];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i0 + i < kRows && ((i0 + i + 1) * kStep <= kTile || r0 + (i0 + i) * kStep < kTile)) {
                const uint32_t to = dst + place_of[i & 3] + (i0 + i) * (kStep * 128);
                if (all) cp16(to, pool + from[i], 16);
                else cp16(to, pool + (from[i] < 0 ? 0 : from[i]), from[i] < 0 ? 0 : 16);
              }
          }
        }
        cp_arrive(&sh.full[slot]);
        if (++slot == kSlots) {
          slot = 0;
          ++turn;
        }
      }
      if (last) break;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // no copy is under way when the block leaves
  } else if (warp == 11) {
    // ---- the products ------------------------------------------------------
    {
      const uint32_t ring = smem_addr(smem), q_at = smem_addr(q_s), p_at = smem_addr(p_s);
      const uint32_t s_col[2] = {tmem, tmem + N}, o_col = tmem + 2 * N;
      int k_idx = 0, items = 0;
      Walk<N> ahead(a, plan);  // the tile whose scores are issued next
      bool more = ahead.next();
      int ahead_tile = more ? ahead.tile0 : 0;
      auto scores = [&]() {  // S^T of the tile `ahead`
        if (ahead_tile == ahead.tile0) wait(&sh.q_full, items++ & 1);
        const int buf = k_idx & 1, slot = (2 * k_idx) % kSlots;
        wait(&sh.full[slot], ((2 * k_idx) / kSlots) & 1);
        if (k_idx >= 2) wait(&sh.s_free[buf], ((k_idx >> 1) - 1) & 1);
        async_fence();  // the loaders' copies, to the products
        tc_after();
        const uint32_t k_at = ring + slot * L::kSlot;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t in = (ks & 3) * 32, half = ks >> 2;
          tc_mma(s_col[buf], operand(k_at + half * kHalf + in, 16, 1024, 2),
                 operand(q_at + half * (N * 128) + in, 16, 1024, 2), instruction<N>(false, false), ks > 0);
        }
        tc_commit(&sh.s_full[buf]);
        tc_commit(&sh.empty[slot]);
        ++k_idx;
        if (++ahead_tile == ahead.tile1) {
          more = ahead.next();
          if (more) ahead_tile = ahead.tile0;
        }
      };
      if (more) scores();
      int v_idx = 0;
      while (at.next()) {
        for (int tile = at.tile0; tile < at.tile1; ++tile, ++v_idx) {
          // the next item's queries come after this item's last weights
          const bool next_item = ahead_tile == ahead.tile0;
          if (more && !next_item) scores();
          const int slot = (2 * v_idx + 1) % kSlots;
          wait(&sh.full[slot], ((2 * v_idx + 1) / kSlots) & 1);
          wait(&sh.p_full, v_idx & 1);
          async_fence();
          tc_after();
          const uint32_t v_at = ring + slot * L::kSlot;
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
              tc_mma(o_col, operand(v_at + ks * 2048, kHalf, 1024, 2),
                     operand(p_at + part * L::kP + ks * 256, 128, 2048, 0), instruction<N>(true, true),
                     tile > at.tile0 || part > 0 || ks > 0);
          tc_commit(&sh.empty[slot]);
          tc_commit(&sh.p_free);
          if (more && next_item) scores();
        }
      }
    }
    __syncwarp();
  } else {
    // ---- softmax: one token and half of the rows a thread ----------------------
    constexpr int kHalfN = N / 2;
    const int group = warp >> 2, quad = warp & 3, token = tid & (kTile - 1), row_a = group * kHalfN;
    const uint32_t lanes = (static_cast<uint32_t>(quad * 32) << 16) + row_a;  // this warp's TMEM lanes, its group's columns
    const uint32_t s_col[2] = {tmem + lanes, tmem + N + lanes}, o_col = tmem + 2 * N + lanes;
    const int G = a.Hq / a.cache.heads;
    auto load_q = [&](const Walk<N>& x) {
      for (int r = tid; r < N; r += kSoft) {
        const AttnRow ar = attn_row(a, x.row0 + min(r, x.rows - 1), x.h);
        sh.q_off[r] = x.b * a.q_batch + ar.i * a.q_token + ar.hq * a.q_head;
      }
      soft_sync();
      for (int e = tid; e < N * kChunks; e += kSoft) {
        const int r = e / kChunks, c = e % kChunks;
        uint4 v = __ldg(reinterpret_cast<const uint4*>(a.q + sh.q_off[r] + c * 16));
        if (r >= x.rows) v = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(q_s + (c >> 3) * (N * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
      }
      async_fence();
      mbar_arrive(&sh.q_full);
    };
    Walk<N> ahead(a, plan);  // the item whose queries are loaded next
    if (ahead.next()) load_q(ahead);
    int tile_no = 0;
    while (at.next()) {
      // (the last item's readers of these are done: soft_sync in its finish)
      for (int r = tid; r < N; r += kSoft) {
        sh.m[r] = -INFINITY;
        sh.limit[r] = at.n - a.Q + min(at.row0 + r, at.R - 1) / G;
      }
      if (tid == 0) sh.odd = 0;
      float l[kHalfN];
#pragma unroll
      for (int r = 0; r < kHalfN; ++r) l[r] = 0.f;
      soft_sync();
      for (int tile = at.tile0; tile < at.tile1; ++tile, ++tile_no) {
        const int buf = tile_no & 1, t = tile * kTile + token;
        wait(&sh.s_full[buf], (tile_no >> 1) & 1);
        tc_after();
        const uint32_t* valid = sh.valid[tile_no & 7];
        const bool exists = (valid[quad] >> lane) & 1;
        // a tile whose tokens all exist and are seen by every row needs no mask
        const bool masked =
            tile * kTile + kTile - 1 > at.n - a.Q || (valid[0] & valid[1] & valid[2] & valid[3]) != 0xffffffffu;
        auto score = [&](float x, int r) {
          x *= a.scale_log2;
          return masked && (!exists || t > sh.limit[r]) ? -INFINITY : x;
        };
        bool grow = false;
#pragma unroll
        for (int c = 0; c < kHalfN; c += 8) {
          float s[8];
          tmem_ld8(s, s_col[buf] + c);
#pragma unroll
          for (int i = 0; i < 8; ++i) grow |= score(s[i], row_a + c + i) > sh.m[row_a + c + i] + kSlackT;
        }
        if (group_any(group, grow)) {
          // new reference maxima, and what has been summed so far by them
#pragma unroll
          for (int c = 0; c < kHalfN; c += 8) {
            float s[8];
            tmem_ld8(s, s_col[buf] + c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float x = score(s[i], row_a + c + i);
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
              if (lane == i) sh.wmax[quad][row_a + c + i] = x;
            }
          }
          group_sync(group);
          if (token < kHalfN) {
            const int r = row_a + token;
            const float old = sh.m[r];
            float m = old;
#pragma unroll
            for (int w = 0; w < 4; ++w) m = fmaxf(m, sh.wmax[w][r]);
            if (!(m > old + kSlackT)) m = old;  // (this row's own scores decide)
            sh.m[r] = m;
            sh.corr[r] = old == -INFINITY ? 0.f : ex2(old - m);
          }
          group_sync(group);
          if (tile > at.tile0) {
#pragma unroll
            for (int r = 0; r < kHalfN; ++r) l[r] *= sh.corr[row_a + r];
            wait(&sh.p_free, (tile_no - 1) & 1);  // O^T is complete
            tc_after();
#pragma unroll
            for (int c = 0; c < kHalfN; c += 8) {
              float o[8];
              tmem_ld8(o, o_col + c);
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] *= sh.corr[row_a + c + i];
              tmem_st8(o_col + c, o);
            }
            tmem_st_done();
          }
        }
        if (tile_no > 0) wait(&sh.p_free, (tile_no - 1) & 1);  // P^T has been read
        // A value that is not finite would reach rows that do not see its token
        // as 0 * inf: such values are zero in the product, and added to the
        // rows that see them at the end.  (Tokens that do not exist are
        // zero-filled.)
        if (masked && group == 0 && t > at.n - a.Q) {
          const int slot = (2 * tile_no + 1) % kSlots;
          wait(&sh.full[slot], ((2 * tile_no + 1) / kSlots) & 1);
          uint4* v = reinterpret_cast<uint4*>(smem + slot * L::kSlot + token * 128);
          uint32_t odd = 0;
#pragma unroll 4
          for (int c = 0; c < kChunks; ++c) {
            uint4* piece = v + (c >> 3) * (kHalf / 16) + ((c ^ token) & 7);  // (in an order without bank conflicts)
            const uint4 x = *piece;
            uint32_t u[4] = {x.x, x.y, x.z, x.w}, bad = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (nonfinite2(u[i])) {
                bad = 1;
                if ((u[i] & 0x7f80u) == 0x7f80u) u[i] &= 0xffff0000u;
                if ((u[i] & 0x7f800000u) == 0x7f800000u) u[i] &= 0xffffu;
              }
            if (bad) *piece = make_uint4(u[0], u[1], u[2], u[3]);
            odd |= bad;
          }
          if (odd) sh.odd = 1;
        }
#pragma unroll
        for (int c = 0; c < kHalfN; c += 8) {
          float s[8];
          tmem_ld8(s, s_col[buf] + c);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            float p[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float m = sh.m[row_a + c + i + y];
              p[y] = ex2(score(s[i + y], row_a + c + i + y) - (m == -INFINITY ? 0.f : m));
              l[c + i + y] += p[y];
            }
            hi[i / 2] = pack2(p[0], p[1]);
            lo[i / 2] = pack2(p[0] - bf16_lo(hi[i / 2]), p[1] - bf16_hi(hi[i / 2]));
          }
          char* to = p_s + (row_a + c) / 8 * (kTile * 16) + token * 16;
          *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(to + L::kP) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        async_fence();
        tc_before();
        mbar_arrive(&sh.s_free[buf]);
        mbar_arrive(&sh.p_full);
      }
      // ---- the item, or this block's part of it ---------------------------------
      if (ahead.next()) load_q(ahead);  // its last scores are done: s_full has come
      // sums over the tokens: a butterfly that halves the rows with the lanes
#pragma unroll
      for (int c = 0; c < kHalfN; c += 32) {
        constexpr int kMost = kHalfN < 32 ? (kHalfN < 16 ? 8 : (kHalfN <= 16 ? 16 : 32)) : 32;
        float v[kMost];
#pragma unroll
        for (int i = 0; i < kMost; ++i) v[i] = c + i < kHalfN ? l[c + i < kHalfN ? c + i : 0] : 0.f;
        // lanes beyond kMost rows: plain sums first
#pragma unroll
        for (int o = 16; o >= kMost; o >>= 1)
#pragma unroll
          for (int i = 0; i < kMost; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
#pragma unroll
        for (int o = kMost / 2; o > 0; o >>= 1)
#pragma unroll
          for (int i = 0; i < o; ++i) {
            const float give = (lane & o) ? v[i] : v[i + o], keep = (lane & o) ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        if (lane < kMost && c + lane < kHalfN) sh.lsum[quad][row_a + c + lane] = v[0];
      }
      wait(&sh.p_free, (tile_no - 1) & 1);
      tc_after();
      soft_sync();
      const bool whole = at.whole();
      float* slot = attn_slot<N, D>(a, blockIdx.x, at.tile0 == 0);
      for (int r = tid; r < at.rows; r += kSoft) {
        const float sum = sh.lsum[0][r] + sh.lsum[1][r] + sh.lsum[2][r] + sh.lsum[3][r], m = sh.m[r];
        if (whole) {
          const AttnRow ar = attn_row(a, at.row0 + r, at.h);
          const size_t to = (static_cast<size_t>(at.b) * a.Q + ar.i) * a.Hq + ar.hq;
          sh.out_at[r] = static_cast<long long>(to);
          sh.inv[r] = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
          if (a.lse) a.lse[to] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
        } else {
          slot[N * D + r] = m;
          slot[N * D + N + r] = sum;
        }
      }
      // O^T through shared memory (P^T's place), a row's D values together
      float* o_s = reinterpret_cast<float*>(p_s);
      const int d = token;
      const bool odd = sh.odd;
#pragma unroll 1
      for (int c = 0; c < kHalfN; c += 8) {
        float o[8];
        tmem_ld8(o, o_col + c);
        if (odd) {
          for (int t = max(at.tile0 * kTile, at.n - a.Q + 1); t < min(at.tile1 * kTile, at.n); ++t) {
            const int entry = static_cast<int>(by_page(static_cast<unsigned long long>(t)));
            const int page = a.table.ids[at.b * a.table.stride + entry];
            if (page < 0 || page >= a.cache.pages) continue;
            const float v = load_one<BF16>(a.cache.v + page * a.cache.page_stride +
                                               (t - entry * a.cache.page_size) * a.cache.token_stride + at.h * (D * 2), d);
            if (!isfinite(v))
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (t <= sh.limit[row_a + c + i]) o[i] += v;
          }
        }
#pragma unroll
          for (int i = 0; i < 8; ++i) o_s[(row_a + c + i) * D + d] = o[i];
      }
      soft_sync();
      for (int e = tid; e < at.rows * (D / 4); e += kSoft) {
        const int r = e / (D / 4), x = (e % (D / 4)) * 4;
        float4 v = *reinterpret_cast<const float4*>(o_s + r * D + x);
        if (whole) {
          const float inv = sh.inv[r];
          store4(a.out, sh.out_at[r] * D + x, true, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
        } else {
          *reinterpret_cast<float4*>(slot + r * D + x) = v;
        }
      }
      if (!whole) {
        const long long c0 = at.first() / at.per, c1 = (at.first() + at.tiles - 1) / at.per;
        soft_sync();
        if (tid == 0) {
          __threadfence();
          const bool last = atom_add_acq_rel_gpu(&a.counters[c0], 1u) + 1u == static_cast<unsigned int>(c1 - c0 + 1);
          if (last) a.counters[c0] = 0u;
          sh.last = last;
        }
        soft_sync();
        if (sh.last) attn_join<N, D, kSoft>(a, at.b, at.h, at.row0, at.rows, at.first(), at.tiles, at.per);
      }
      tc_before();  // O^T has been read
      soft_sync();
    }
  }
  tc_before();
  __syncthreads();
  if (warp == 11) {
    tc_after();
    if (*reinterpret_cast<volatile int*>(&sh.dead)) {
      // a wait ran out, so products may be under way: none may be when TMEM is freed and the block leaves
      tc_commit(&sh.done);
      mbar_wait_sleep(&sh.done, 0);
    }
    tmem_free(tmem, L::kCols);
  }
}

template <int N>
cudaError_t prepare() {
  return cudaFuncSetAttribute(attention_tc_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<N>::kBytes);
}
template <int N>
void launch(const AttnArgs& a, int grid, cudaStream_t stream) {
  attention_tc_kernel<N><<<grid, kThreadsT, Lay<N>::kBytes, stream>>>(
      a, DivU64::make(static_cast<unsigned long long>(a.cache.page_size)));
}

}  // namespace tc
}  // namespace specv
