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
// One block per SM.  Warps 0-3 and 4-7: the streams' softmax.  Warps 8 and 9 copy K
// and V of the tiles into a ring of slots, across item boundaries, in 16-byte
// pieces that arrive on the slot's barrier by themselves, so any page size and
// strides.  Warp 10 issues the scores' products, warp 11 the outputs'.
#pragma once

#include "attention_common.cuh"
#include "attention_mma.cuh"
#include "attention_tc.cuh"
#include "tree_common.cuh"

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
using tc::tc_mma;
using tc::tmem_alloc;
using tc::tmem_free;
using tc::tmem_st_done;

constexpr int kTile = 64;        // tokens
constexpr int kSoft = 256;       // softmax threads, 128 a stream
constexpr int kLoad = 64;        // loader threads
constexpr int kThreadsR = kSoft + kLoad + 64;
constexpr float kSlackR = 8.f;   // how far (log2) a score may pass the reference
constexpr int kEndR = 6;         // steps that an item's start and end count as
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
  static constexpr int kBytes = kSlots * kSlot + kQ + 1024;  // 1024: alignment
  static_assert(kSlots >= 8 && kSlots / 2 + 4 < kAhead, "the ring");
};

template <int D, bool kDual>
struct Shared {
  unsigned long long full[Lay<D, kDual>::kSlots], empty[Lay<D, kDual>::kSlots];
  unsigned long long s_full[2][2], p_full[2][2], pv_done[2][2], q_full[2] /* one for both streams of shared rows */, done[2];
  long long off[2][kTile];    // byte offsets of a tile's tokens, -1: none
  uint32_t valid[kAhead][2];  // tokens that exist, by tile
  long long q_off[2][128];    // of the next item's rows, bytes
  TreeSight<128> sight[2];
  float m[2][128], l[2][128];
  int odd[kOdd];              // the item has values that are not finite and not every row sees
  uint32_t tmem;
  int dead;                   // a wait ran out: nothing waits any more
  int last;
  long long plan[2 * (kThreadsR / 32) + 4];
};

// O += P V with P in TMEM.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
      : "memory");
}
#define SPEC_R8(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]), "=r"(x[i + 5]), "=r"(x[i + 6]), "=r"(x[i + 7])
#define SPEC_I8(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])
// 32 columns of the warp's lanes (the wait in the same statement: no use comes before it).
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
__device__ __forceinline__ void st32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::SPEC_I8(r, 0), SPEC_I8(r, 8), SPEC_I8(r, 16), SPEC_I8(r, 24), "r"(at)
      : "memory");
}
#undef SPEC_R8
#undef SPEC_I8

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ void load_sync() { asm volatile("bar.sync 2, 64;" ::: "memory"); }
__device__ __forceinline__ void stream_sync(int s) { asm volatile("bar.sync %0, 128;" ::"r"(3 + s) : "memory"); }

template <int D, bool kDual>
__global__ void __launch_bounds__(kThreadsR, 1) attention_tree_kernel(const AttnArgs a, DivU64 by_page) {
  using L = Lay<D, kDual>;
  using Walk = AttnWalk<kTile, kEndR, L::kRows>;
  constexpr int kSlots = L::kSlots, kHalf = L::kHalf, kChunks = D / 8;  // 16-byte pieces of a token
  constexpr int kCols = 512, kStream = 256, kO = 128;                   // TMEM: a stream's S / P buffers, then its O
  extern __shared__ char raw_smem[];
  __shared__ Shared<D, kDual> sh;
  char* smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  char* q_s = smem + kSlots * L::kSlot;  // [128-row tiles][halves][128][128 bytes]
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

  const AttnPlan plan = attn_plan<kTile, kEndR, kThreadsR>(
      a, a.cache.heads * ((a.Q * (a.Hq / a.cache.heads) + L::kRows - 1) / L::kRows), 4, sh.plan);
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sh.full[i], kLoad + 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sh.s_full[s][i], 1);
        mbar_init(&sh.p_full[s][i], 4);
        mbar_init(&sh.pv_done[s][i], 1);
      }
      mbar_init(&sh.q_full[s], 128);
      mbar_init(&sh.done[s], 1);
    }
    for (int i = 0; i < kOdd; ++i) sh.odd[i] = 0;
    sh.dead = 0;
    fence_barrier_init();
  }
  if (warp == 11) tmem_alloc(&sh.tmem, kCols);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = sh.tmem;
  Walk at(a, plan);

  if (warp == 8 || warp == 9) {
    // ---- K and V of each tile, in turn -----------------------------------
    const int lt = tid - kSoft, S = a.cache.page_size;
    const int chunk = lt % kChunks, r0 = lt / kChunks;
    constexpr int kStep = kLoad / kChunks, kPasses = kTile / kStep;
    // The tile whose pages are looked up, one ahead of the copies: the table's
    // entries are on their way while the tile before is copied.
    Walk ahead(a, plan);
    bool more = ahead.next();
    int ahead_tile = more ? ahead.tile0 : 0;
    int page, place, head = 0;  // place: token in the page, -1: past the end
    auto look_up = [&]() {
      head = ahead.h;
      const int t = ahead_tile * kTile + lt;
      const int entry = static_cast<int>(by_page(static_cast<unsigned long long>(t)));
      place = t < ahead.n ? t - entry * S : -1;
      page = t < ahead.n ? __ldg(a.table.ids + ahead.b * a.table.stride + entry) : -1;
      if (++ahead_tile == ahead.tile1) {
        more = ahead.next();
        if (more) ahead_tile = ahead.tile0;
      }
    };
    const bool any = more;
    if (any) look_up();
    uint32_t place_of[2];  // where the thread's piece of row r0 + i * kStep lies in the swizzled slot
#pragma unroll
    for (int i = 0; i < 2; ++i)
      place_of[i] = (chunk >> 3) * kHalf + r0 * 128 + (((chunk & 7) ^ ((r0 + i * kStep) & 7)) << 4);
    static_assert(2 * kStep % 8 == 0, "two passes go round");
    int slot = 0;
    uint32_t turn = 0;  // times the ring went round
    for (int tile_no = 0; any; ++tile_no) {
      const bool ok = page >= 0 && page < a.cache.pages;
      if (!ok && place >= 0 && a.status) atomicOr(a.status, kDataPageRange);
      const uint32_t exists = __ballot_sync(0xffffffffu, ok);
      if (lane == 0) sh.valid[tile_no % kAhead][warp - 8] = exists;
      sh.off[tile_no & 1][lt] = ok ? page * a.cache.page_stride + place * a.cache.token_stride + head * (D * 2) : -1ll;
      load_sync();
      const bool last = !more;
      if (more) look_up();
      const uint32_t* valid = sh.valid[tile_no % kAhead];
      const bool all = (valid[0] & valid[1]) == 0xffffffffu;
      const long long* off = sh.off[tile_no & 1] + r0;
#pragma unroll 1
      for (int x = 0; x < 2; ++x) {
        if (turn > 0) wait(&sh.empty[slot], (turn + 1) & 1);
        const char* pool = (x ? a.cache.v : a.cache.k) + chunk * 16;
        const uint32_t dst = smem_addr(smem) + slot * L::kSlot;
#pragma unroll
        for (int i0 = 0; i0 < kPasses; i0 += 8) {  // (offsets are read ahead of the copies, which no load passes)
          long long from[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) from[i] = off[(i0 + i) * kStep];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t to = dst + place_of[i & 1] + (i0 + i) * (kStep * 128);
            if (all) cp16(to, pool + from[i], 16);
            else cp16(to, pool + (from[i] < 0 ? 0 : from[i]), from[i] < 0 ? 0 : 16);
          }
        }
        cp_arrive(&sh.full[slot]);
        if (lt == 0) mbar_arrive(&sh.full[slot]);  // (the tile's bits, stored before load_sync, come with it)
        if (++slot == kSlots) {
          slot = 0;
          ++turn;
        }
      }
      if (last) break;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // no copy is under way when the block leaves
  } else if (warp == 10) {
    // ---- scores ----------------------------------------------------------------
    const uint32_t ring = smem_addr(smem), q_at = smem_addr(q_s);
    int count[2] = {0, 0}, tile_no = 0, items = 0;
    while (at.next()) {
      for (int tile = at.tile0; tile < at.tile1; ++tile, ++tile_no) {
        const int slot = (2 * tile_no) % kSlots;
        wait(&sh.full[slot], ((2 * tile_no) / kSlots) & 1);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!kDual && s != ((tile - at.tile0) & 1)) continue;
          const int c = count[s]++, buf = c & 1;
          if (tile == at.tile0) wait(&sh.q_full[s], items & 1);
          if (c >= 2) wait(&sh.pv_done[s][buf], ((c >> 1) - 1) & 1);
          async_fence();  // the copies, to the products
          tc_after();
          const uint32_t k_at = ring + slot * L::kSlot, qs = q_at + (kDual ? s : 0) * (128 * D * 2);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t in = (ks & 3) * 32, half = ks >> 2;
            tc_mma(tmem + s * kStream + buf * kTile, operand(qs + half * (128 * 128) + in, 16, 1024, 2),
                   operand(k_at + half * kHalf + in, 16, 1024, 2), tc::instruction<kTile>(false, false), ks > 0);
          }
          if (!kDual || s == 1) tc_commit(&sh.empty[slot]);
          tc_commit(&sh.s_full[s][buf]);
        }
      }
      ++items;
    }
    if (*reinterpret_cast<volatile int*>(&sh.dead)) {  // none of them may be under way when TMEM is freed
      tc_commit(&sh.done[0]);
      mbar_wait_sleep(&sh.done[0], 0);
    }
    __syncwarp();
  } else if (warp == 11) {
    // ---- outputs -----------------------------------------------------------------
    const uint32_t ring = smem_addr(smem);
    int count[2] = {0, 0}, tile_no = 0;
    while (at.next()) {
      for (int tile = at.tile0; tile < at.tile1; ++tile, ++tile_no) {
        const int slot = (2 * tile_no + 1) % kSlots;
        wait(&sh.full[slot], ((2 * tile_no + 1) / kSlots) & 1);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!kDual && s != ((tile - at.tile0) & 1)) continue;
          const int c = count[s]++, buf = c & 1;
          wait(&sh.p_full[s][buf], (c >> 1) & 1);
          async_fence();
          tc_after();
          const uint32_t v_at = ring + slot * L::kSlot, p = tmem + s * kStream + buf * kTile;
          const bool first = kDual ? tile == at.tile0 : tile - at.tile0 < 2;
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
              tc_mma_ts(tmem + s * kStream + kO, p + part * (kTile / 2) + ks * 8, operand(v_at + ks * 2048, kHalf, 1024, 2),
                        tc::instruction<D>(false, true), !first || part > 0 || ks > 0);
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
  } else {
    // ---- softmax: a row a thread --------------------------------------------------
    const int s = warp >> 2, row_in = tid & 127, quad = warp & 3;
    const int row_at = kDual ? s * 128 : 0;  // the stream's first row of an item
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_col = tmem + lanes + s * kStream, o_col = s_col + kO;
    const float scale = fabsf(a.scale_log2) > 0.f ? fabsf(a.scale_log2) : 1.f;
    const bool turned = !(a.scale_log2 > 0.f), flat = a.scale_log2 == 0.f;  // scores change their sign; are all zero
    TreeSight<128>& sight = sh.sight[s];
    auto load_q = [&](const Walk& x) {  // under way when it returns
      stream_sync(s);  // (q_off is free)
      {
        const AttnRow ar = attn_row(a, x.row0 + min(row_at + row_in, x.rows - 1), x.h);
        sh.q_off[s][row_in] = x.b * a.q_batch + ar.i * a.q_token + ar.hq * a.q_head;
      }
      stream_sync(s);
      const uint32_t to = smem_addr(q_s) + (kDual ? s : 0) * (128 * D * 2);
#pragma unroll 4
      for (int e = row_in; e < 128 * kChunks; e += 128) {
        const int r = e / kChunks, c = e % kChunks;
        cp16(to + (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4), a.q + sh.q_off[s][r] + c * 16,
             row_at + r < x.rows ? 16 : 0);
      }
    };
    auto q_loaded = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      async_fence();
      mbar_arrive(&sh.q_full[kDual ? s : 0]);
    };
    Walk ahead(a, plan);  // the item whose queries are loaded next
    bool more = ahead.next();
    if (more && (kDual || s == 0)) {
      load_q(ahead);
      q_loaded();
    }
    if (more) more = ahead.next();
    int count = 0, tile_no = 0, items = 0, sight_b = -1, sight_rt = -1;
    while (at.next()) {
      const int base = at.n - a.Q;
      if (at.b != sight_b || at.rt != sight_rt) {
        stream_sync(s);
        tree_sight<128>(a, at.b, base, at.row0 + row_at, at.row0 + at.rows - 1, row_in, 128, sight, [&] { stream_sync(s); });
        sight_b = at.b;
        sight_rt = at.rt;
      }
      if (tid == 0) sh.odd[(items + kOdd / 2) % kOdd] = 0;
      float m = -INFINITY, l = 0.f;
      const int tiles = at.tile1 - at.tile0;
      const int first = kDual ? 0 : s, step = kDual ? 1 : 2;
      for (int j = first; j < tiles; j += step, ++count) {
        const int tile = at.tile0 + j, buf = count & 1, t0 = tile * kTile, now = tile_no + j;
        wait(&sh.s_full[s][buf], (count >> 1) & 1);
        tc_after();
        const bool last = j == tiles - 1;  // the item's last scores are done, so its queries have been read
        if (last && more) load_q(ahead);
        uint32_t x[64];
        ld64(x, s_col + buf * kTile);
        if (turned) {
#pragma unroll
          for (int i = 0; i < 64; ++i) x[i] = flat ? 0u : x[i] ^ 0x80000000u;
        }
        const uint32_t* valid = sh.valid[now % kAhead];
        const uint32_t v0 = valid[0], v1 = valid[1];
        // a tile whose tokens all exist and come before the tree needs no mask
        if ((v0 & v1) != 0xffffffffu || t0 + kTile > base) {
          const uint32_t see[2] = {v0 & sight.window(row_in, t0 - base), v1 & sight.window(row_in, t0 + 32 - base)};
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (!((see[i >> 5] >> (i & 31)) & 1)) x[i] = 0xff800000u;  // -inf
          // A value that is not finite would reach rows that do not see its token
          // as 0 * inf: such values are zero in the products, and added to the
          // rows that see them at the end.  (Tokens that do not exist are
          // zero-filled.  The first stream does it for both: the second's
          // products with the tile are issued after the first's.)
          if (t0 + kTile > base && (!kDual || s == 0)) {
            const int slot = (2 * now + 1) % kSlots;
            wait(&sh.full[slot], ((2 * now + 1) / kSlots) & 1);
            const int token = row_in & (kTile - 1);
            constexpr int kPer = kChunks / 2;  // pieces a thread looks at
            if (t0 + token >= base) {
              uint4* v = reinterpret_cast<uint4*>(smem + slot * L::kSlot + token * 128);
              bool odd = false;
#pragma unroll
              for (int i = 0; i < kPer; ++i) {
                const int c = (row_in >> 6) * kPer + i;
                uint4* piece = v + (c >> 3) * (kHalf / 16) + ((c ^ token) & 7);  // (in an order without bank conflicts)
                const uint4 w = *piece;
                uint32_t u[4] = {w.x, w.y, w.z, w.w};
                bool bad = false;
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  if (nonfinite2(u[y])) {
                    bad = true;
                    if ((u[y] & 0x7f80u) == 0x7f80u) u[y] &= 0xffff0000u;
                    if ((u[y] & 0x7f800000u) == 0x7f800000u) u[y] &= 0xffffu;
                  }
                if (bad) *piece = make_uint4(u[0], u[1], u[2], u[3]);
                odd |= bad;
              }
              if (odd) {
                sh.odd[items % kOdd] = 1;
                async_fence();
              }
            }
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 64; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(x[i]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
        const bool grow = top > m + kSlackR;
        if (__any_sync(0xffffffffu, grow)) {
          const float c = grow ? (m == -INFINITY ? 0.f : ex2(m - top)) : 1.f;
          if (grow) m = top;
          if (j > first) {
            l *= c;
            wait(&sh.pv_done[s][buf ^ 1], ((count - 1) >> 1) & 1);  // O is complete
            tc_after();
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
              uint32_t o[32];
              ld32(o, o_col + d);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * c);
              st32(o_col + d, o);
            }
          }
        }
        const float less = m == -INFINITY ? 0.f : -m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t hi[32], lo[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float p0 = ex2(fmaf(__uint_as_float(x[2 * i]), scale, less));
          const float p1 = ex2(fmaf(__uint_as_float(x[2 * i + 1]), scale, less));
          sum[(2 * i) & 3] += p0;
          sum[(2 * i + 1) & 3] += p1;
          hi[i] = pack2(p0, p1);
          lo[i] = pack2(p0 - bf16_lo(hi[i]), p1 - bf16_hi(hi[i]));
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        st32(s_col + buf * kTile, hi);
        st32(s_col + buf * kTile + 32, lo);
        tmem_st_done();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[s][buf]);
        if (last && more) q_loaded();
      }
      if (more) more = ahead.next();

      // ---- the item, or this block's part of it ---------------------------------
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
      const int r = row_at + row_in;  // of the item
      const bool row = r < at.rows, none = sight.blind(row_in);
      if (none) {  // no node: what it summed over the context is nobody's
        m = -INFINITY;
        l = 0.f;
      }
      const AttnRow ar = attn_row(a, at.row0 + min(r, at.rows - 1), at.h);
      const size_t to = (static_cast<size_t>(at.b) * a.Q + ar.i) * a.Hq + ar.hq;
      float* slot = attn_slot<L::kRows, D>(a, blockIdx.x, at.tile0 == 0);
      const float inv = whole ? (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) : 1.f;
      const bool odd = *reinterpret_cast<volatile int*>(&sh.odd[items % kOdd]) != 0;
      constexpr int kPart = kDual ? D : D / 2;  // columns that the thread writes
#pragma unroll 1
      for (int d = kDual ? 0 : s * kPart; d < (kDual ? D : (s + 1) * kPart); d += 32) {
        uint32_t u[32];
        float o[32];
        ld32(u, tmem + lanes + (kDual ? s * kStream : 0) + kO + d);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(u[i]);
        if constexpr (!kDual) {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= c0;
          if (both) {
            ld32(u, tmem + lanes + kStream + kO + d);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = fmaf(c1, __uint_as_float(u[i]), o[i]);
          }
        }
        if (odd) {
          for (int t = max(at.tile0 * kTile, max(base, 0)); t < min(at.tile1 * kTile, at.n); ++t) {
            if (!sight.sees(row_in, t - base)) continue;
            const int entry = static_cast<int>(by_page(static_cast<unsigned long long>(t)));
            const int page = a.table.ids[at.b * a.table.stride + entry];
            if (page < 0 || page >= a.cache.pages) continue;
            const char* v = a.cache.v + page * a.cache.page_stride + (t - entry * a.cache.page_size) * a.cache.token_stride +
                            at.h * (D * 2);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float y = load_one<BF16>(v, d + i);
              if (!isfinite(y)) o[i] += y;
            }
          }
        }
        if (!row) continue;
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = none ? 0.f : o[i] * inv;
        if (whole) {
          uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + to * D + d);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            out[i] = make_uint4(pack2(o[8 * i], o[8 * i + 1]), pack2(o[8 * i + 2], o[8 * i + 3]), pack2(o[8 * i + 4], o[8 * i + 5]),
                                pack2(o[8 * i + 6], o[8 * i + 7]));
        } else {
          float4* out = reinterpret_cast<float4*>(slot + r * D + d);
#pragma unroll
          for (int i = 0; i < 8; ++i) out[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
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
      if (!whole) {
        soft_sync();
        if (tid == 0) {
          const long long k0 = at.first() / at.per, k1 = (at.first() + at.tiles - 1) / at.per;
          __threadfence();
          const bool last = atom_add_acq_rel_gpu(&a.counters[k0], 1u) + 1u == static_cast<unsigned int>(k1 - k0 + 1);
          if (last) a.counters[k0] = 0u;
          sh.last = last;
        }
        soft_sync();
        if (sh.last) attn_join<L::kRows, D, kSoft>(a, at.b, at.h, at.row0, at.rows, at.first(), at.tiles, at.per);
        soft_sync();
      } else if constexpr (!kDual) {
        soft_sync();  // both streams' O may be written again
      }
      tile_no += tiles;
      ++items;
    }
  }
  tc_before();
  __syncthreads();
  if (warp == 11) {
    tc_after();
    tmem_free(tmem, kCols);
  }
}

template <int D, bool kDual>
cudaError_t prepare() {
  return cudaFuncSetAttribute(attention_tree_kernel<D, kDual>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D, kDual>::kBytes);
}
template <int D, bool kDual>
void launch(const AttnArgs& a, int sm_count, cudaStream_t stream) {
  attention_tree_kernel<D, kDual><<<sm_count < kMaxCtas ? sm_count : kMaxCtas, kThreadsR, Lay<D, kDual>::kBytes, stream>>>(
      a, DivU64::make(static_cast<unsigned long long>(a.cache.page_size)));
}

}  // namespace ttc
}  // namespace specv
