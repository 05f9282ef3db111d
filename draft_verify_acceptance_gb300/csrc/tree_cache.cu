// tree_cache.cu -- the cache's side of speculation over trees: appending with
// the position rotation applied, accepting a path, keeping its tokens (sm_103a).
#include <climits>

#include "device_common.cuh"
#include "launch_tree.h"
#include "tree_common.cuh"

namespace specv {
namespace {

__device__ __forceinline__ void report(int32_t* status, int bits) {
  if (bits && status) atomicOr(status, bits);
}

// ---- rotated append ----------------------------------------------------------
// (x, y) -> (x cos a - y sin a, y cos a + x sin a),  a = position * inv_freq.
//
// Turns per position are a 64-bit binary fraction, so that position * turns is
// exact modulo one turn however far the position is: a product of the frequency's
// 24-bit significand and 1 / (2 pi), shifted by its exponent, all in integers.
// It is within two of its last places up to frequencies of 1, where 64 bits of
// 1 / (2 pi) do.  A higher one needs bits further down (Payne and Hanek, 1983: of m * 2^k / (2 pi)
// only the bits of 1 / (2 pi) from the k-th on reach the fraction), and is within one.
__constant__ const uint32_t kInv2PiWords[7] = {  // the first 224 bits of 1 / (2 pi)
    0x28be60dbu, 0x9391054au, 0x7f09d5f4u, 0x7d4d3770u, 0x36d8a566u, 0x4f10e410u, 0x7f9458eau};
// Of m * 2^k, m below 2^24 and k from -23 to 105.  (Rare, and a call of its own: in line, its
// code made 64 trees of 16 take 8.9 us; so they take 8.5, and without it 8.4.)
__device__ __noinline__ unsigned long long turns_of_high(uint32_t m, int k) {
  const int word = k > 0 ? k >> 5 : 0, bit = k > 0 ? k & 31 : 0;
  uint32_t w[3];  // 96 bits from there on
#pragma unroll
  for (int i = 0; i < 3; ++i) w[i] = __funnelshift_l(kInv2PiWords[word + i + 1], kInv2PiWords[word + i], bit);
  const unsigned long long first = static_cast<unsigned long long>(m) * w[0];
  const unsigned long long rest = static_cast<unsigned long long>(m) * w[1] + ((static_cast<unsigned long long>(m) * w[2]) >> 32);
  const unsigned long long lo = rest + (first << 32);
  return k >= 0 ? lo : (lo >> -k) | (((first >> 32) + (lo < rest)) << (64 + k));
}
__device__ __forceinline__ unsigned long long turns_of(float f) {
  constexpr unsigned long long kInv2Pi = 0x28be60db9391054aull;  // 2^64 / (2 pi)
  const uint32_t u = __float_as_uint(f), e = (u >> 23) & 255;
  const unsigned long long m = e ? (u & 0x7fffffu) | 0x800000u : u & 0x7fffffu;
  const int shift = 150 - static_cast<int>(e ? e : 1);  // |f| = m * 2^-shift
  unsigned long long t;
  if ((u & 0x7fffffffu) > 0x3f800000u) {
    t = turns_of_high(static_cast<uint32_t>(m), -shift);
  } else {
    const unsigned long long lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
    if (shift >= 128) t = 0;
    else if (shift >= 64) t = hi >> (shift - 64);
    else t = (lo >> shift) | (hi << (64 - shift));  // (shift is 23 and more)
  }
  return u >> 31 ? 0ull - t : t;
}

// cos and sin of `phase` / 2^32 turns: an eighth of a turn to either side of the
// nearest quarter, there by their power series (cut behind x^9 and x^10: 2^-28
// of them), and the quarters by swaps and signs.
__device__ __forceinline__ float2 cos_sin(uint32_t phase) {
  const uint32_t quarter = (phase + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(phase - (quarter << 30))) * 1.46291807926716e-9f;  // 2 pi / 2^32
  const float z = x * x;
  float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
  s = fmaf(z, s, 8.3333333e-3f);
  s = fmaf(z, s, -1.6666667e-1f);
  s = fmaf(z * x, s, x);
  float c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
  c = fmaf(z, c, -1.3888889e-3f);
  c = fmaf(z, c, 4.1666667e-2f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.f);
  const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
  return make_float2((quarter + 1) & 2 ? -a : a, quarter & 2 ? -b : b);
}

// 16 bytes as floats, and back with one rounding.
template <typename E>
struct Piece {
  static constexpr int kN = 16 / E::kBytes;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&x)[kN]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (E::kBytes == 4) {
        x[i] = __uint_as_float(u[i]);
      } else {
        x[2 * i] = bf16_lo(u[i]);
        x[2 * i + 1] = bf16_hi(u[i]);
      }
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[kN]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (E::kBytes == 4) u[i] = __float_as_uint(x[i]);
      else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

constexpr int kMaxFreq = 128;
constexpr int kAppendWarps = 8;
constexpr int kBatch = 4;  // units, and pieces of the values, that a lane has under way

// Division of indexes below 2^23 by up to 2^8: one multiply-high.
struct Div32 {
  uint32_t m = 0;  // 0: divide by 1
  static Div32 make(int d) {
    Div32 r;
    r.m = d <= 1 ? 0u : static_cast<uint32_t>((1ull << 32) / static_cast<unsigned>(d) + 1);
    return r;
  }
  __device__ __forceinline__ int operator()(int n) const { return m ? static_cast<int>(__umulhi(static_cast<uint32_t>(n), m)) : n; }
};

// 16 bytes that are read once.  (Not by the read-only path: the queries may be rotated in place.)
__device__ __forceinline__ uint4 ld_once(const uint4* p) { return __ldcs(p); }

// A token's queries and keys are units: a piece of 16 bytes of a rotated head and
// the one n_freq dimensions on (interleaved: one piece, its pairs side by side), or
// a piece behind the rotated dimensions; its values are pieces.  `parts` warps share
// a token.  A warp's first units and pieces are under way while it finds the
// token's place and turns its angles, which every part does for itself.  HBM bounds
// many tokens (53141 tokens of 12 prompts, 32 + 8 heads of 128, bf16: 201 us, 97 % of the
// copy rate; one unit at a time it was 219), the dependent look-ups few (64 trees of
// 16: 8.4 us, 25 MB).
template <typename E, bool kInterleaved>
__global__ void __launch_bounds__(kAppendWarps * 32)
rotated_append_kernel(const RotatedAppendArgs a, int parts, DivU64 by_part, Div32 by_unit) {
  constexpr int kN = Piece<E>::kN;
  __shared__ float2 s_turn[kAppendWarps][kMaxFreq];  // of pair p of a unit's pairs, unit u: p * turned + u, so that lanes read side by side
  constexpr int kPairs = kInterleaved ? kN / 2 : kN;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long job = static_cast<long long>(blockIdx.x) * kAppendWarps + warp;
  const int row = static_cast<int>(by_part(static_cast<unsigned long long>(job)));
  const int part = static_cast<int>(job - static_cast<long long>(row) * parts);
  if (row >= a.T) return;
  const int D = a.cache.head_dim, F = a.n_freq, H = a.cache.heads;
  const int turned = kInterleaved ? 2 * F / kN : F / kN, per_head = turned + (D - 2 * F) / kN;
  const int units = (a.q_heads + H) * per_head, q_units = a.q_heads * per_head, pieces = H * (D / kN), stride = parts * 32;
  const char* q = a.q + row * a.q_stride;
  const char* k = a.k_new + row * a.new_stride;
  const uint4* v = reinterpret_cast<const uint4*>(a.v_new + row * a.new_stride);

  uint4 x[kBatch], y[kBatch], w[kBatch];
  auto unit_at = [&](int j, int& u) -> long long {  // byte offset in the queries' or the keys' row
    const int jj = j < q_units ? j : j - q_units, head = by_unit(jj);
    u = jj - head * per_head;
    return static_cast<long long>(head) * (D * E::kBytes);
  };
  auto load = [&](int j0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int j = j0 + i * stride;
      if (j >= units) break;
      int u;
      const long long in = unit_at(j, u);
      const uint4* from = reinterpret_cast<const uint4*>((j < q_units ? q : k) + in);
      x[i] = ld_once(from + (u < turned ? u : 2 * F / kN + u - turned));
      if (!kInterleaved && u < turned) y[i] = ld_once(from + u + turned);
    }
  };
  auto load_v = [&](int j0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (j0 + i * stride < pieces) w[i] = ld_once(v + j0 + i * stride);
  };
  const int j0 = part * 32 + lane;
  load(j0);
  load_v(j0);

  // the token's sequence and place
  int b, after;
  bool claimed = true;
  const int given = a.positions ? a.positions[row] : 0;
  if (a.starts) {
    // the last b with starts[b] <= row, 32 entries at a time
    int lo = 0, n = a.B;
    while (n > 1) {
      const int step = (n + 31) >> 5, i = lo + lane * step;
      const uint32_t below = __ballot_sync(0xffffffffu, lane * step < n && (lane == 0 || a.starts[i] <= row));
      const int last = 31 - __clz(below);
      lo += last * step;
      n = min(step, n - last * step);
    }
    b = lo;
    const int from = a.starts[b], to = a.starts[b + 1];
    after = to - row;
    claimed = from <= row && after > 0 && to <= a.T;
  } else {
    const int per = a.T / a.B;
    b = row / per;
    after = per - (row - b * per);
  }
  const long long place = claimed ? static_cast<long long>(a.lengths[b]) - after : -1;
  const bool in = place >= 0 && place < static_cast<long long>(a.table.max_pages) * a.cache.page_size;
  const int at = static_cast<int>(place), slot = in ? at / a.cache.page_size : 0;
  const int page = in ? a.table.ids[b * a.table.stride + slot] : -1;  // on its way while the angles are turned
  const long long position = a.positions ? given : at;
  for (int i = lane; i < F; i += 32)
    s_turn[warp][i % kPairs * turned + i / kPairs] =
        cos_sin(static_cast<uint32_t>((static_cast<unsigned long long>(position) * turns_of(a.inv_freq[i])) >> 32));
  __syncwarp();
  const bool kept = page >= 0 && page < a.cache.pages;
  if (part == 0 && lane == 0 && !kept) report(a.status, in ? kDataPageRange : kDataLengthRange);
  const long long off = kept ? page * a.cache.page_stride + (at - slot * a.cache.page_size) * a.cache.token_stride : -1;
  char* q_out = a.q_out + row * a.q_out_stride;
  if (!claimed) {
    if (a.q_out != a.q)
      for (int j = j0; j < a.q_heads * (D / kN); j += stride) reinterpret_cast<uint4*>(q_out)[j] = make_uint4(0, 0, 0, 0);
    return;
  }

  if (off >= 0)
    for (int j = j0; j < pieces;) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (j + i * stride < pieces) reinterpret_cast<uint4*>(a.cache.v + off)[j + i * stride] = w[i];
      j += kBatch * stride;
      load_v(j);
    }
  float2 t[kPairs];  // of unit `have`: mostly all of a lane's
  int have = -1;
  for (int j1 = j0; j1 < units;) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int j = j1 + i * stride;
      if (j >= units) break;
      int u;
      const long long in = unit_at(j, u);
      if (j >= q_units && off < 0) continue;
      uint4* to = reinterpret_cast<uint4*>((j < q_units ? q_out : a.cache.k + off) + in);
      if (u >= turned) {
        to[2 * F / kN + u - turned] = x[i];
        continue;
      }
      if (u != have) {
        have = u;
#pragma unroll
        for (int e = 0; e < kPairs; ++e) t[e] = s_turn[warp][e * turned + u];
      }
      float f[kN];
      Piece<E>::unpack(x[i], f);
      if constexpr (kInterleaved) {
#pragma unroll
        for (int e = 0; e < kN; e += 2) {
          const float p = f[e], r = f[e + 1];
          f[e] = p * t[e / 2].x - r * t[e / 2].y;
          f[e + 1] = r * t[e / 2].x + p * t[e / 2].y;
        }
        to[u] = Piece<E>::pack(f);
      } else {
        float g[kN];
        Piece<E>::unpack(y[i], g);
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const float p = f[e], r = g[e];
          f[e] = p * t[e].x - r * t[e].y;
          g[e] = r * t[e].x + p * t[e].y;
        }
        to[u] = Piece<E>::pack(f);
        to[u + turned] = Piece<E>::pack(g);
      }
    }
    j1 += kBatch * stride;
    load(j1);
  }
}

// ---- accept --------------------------------------------------------------------
// One warp a tree, a lane holding nodes lane, lane + 32, ...: a step compares all
// of them with (node, drawn token) and takes the lowest match.  A launch bounds it:
// 512 trees of 64 nodes 6 to 9 us by the host, four trees the same.
constexpr int kAcceptWarps = 4;
__global__ void __launch_bounds__(kAcceptWarps * 32) tree_accept_kernel(const AcceptArgs a) {
  __shared__ int32_t s_drawn[kAcceptWarps][kMaxNodes], s_path[kAcceptWarps][kMaxNodes];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x * kAcceptWarps + warp;
  if (b >= a.B) return;
  const long long row = static_cast<long long>(b) * a.N;
  int parent[kNodeWords], token[kNodeWords];
  bool bad = false;
#pragma unroll
  for (int x = 0; x < kNodeWords; ++x) {
    const int i = x * 32 + lane;
    parent[x] = -2;
    token[x] = 0;
    if (i < a.N) {
      parent[x] = a.parents[b * a.parents_stride + i];
      token[x] = a.tokens[row + i];
      s_drawn[warp][i] = a.drawn[row + i];
      s_path[warp][i] = -1;
      if (parent[x] >= i) {
        bad = true;
        parent[x] = -2;
      }
    }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) report(a.status, kDataTreeParent);
  __syncwarp();
  int n = 0;
  if (__shfl_sync(0xffffffffu, parent[0], 0) == -1) {
    for (int node = 0; node < kMaxNodes;) {
      const int t = s_drawn[warp][node];
      if (lane == 0) s_path[warp][n] = node;
      ++n;
      int next = kMaxNodes;
#pragma unroll
      for (int x = kNodeWords - 1; x >= 0; --x)
        if (parent[x] == node && token[x] == t) next = x * 32 + lane;
      node = __reduce_min_sync(0xffffffffu, next);
    }
  }
  __syncwarp();
  if (lane == 0) a.accepted_len[b] = n - 1;
#pragma unroll
  for (int x = 0; x < kNodeWords; ++x) {
    const int j = x * 32 + lane;
    if (j < a.N) {
      const int node = s_path[warp][j];
      a.path[row + j] = node;
      a.out_tokens[row + j] = node >= 0 ? s_drawn[warp][node] : -1;
    }
  }
}

// ---- keep ------------------------------------------------------------------------
// A thread owns one 16-byte column of a sequence's tokens in one layer of K or V
// and makes the path's moves in order, eight loads under way: a token comes from
// its own index or a later one, so no load of a batch, or of a later one, reads
// what a store of it has written.  64 trees of 64 nodes in 16 layers, 8 heads of 128,
// bf16, 6 nodes moved a tree: 14.1 to 15.7 us (their bytes at the copy rate 11.3).
constexpr int kKeepThreads = 128, kKeepMoves = 128;
__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const KeepArgs a, unsigned chunks) {
  __shared__ long long s_from[kKeepMoves], s_to[kKeepMoves];
  __shared__ int s_end;
  const int tid = threadIdx.x, S = a.cache.page_size;
  const int b = static_cast<int>(blockIdx.x / chunks), chunk = static_cast<int>(blockIdx.x - static_cast<unsigned>(b) * chunks);
  const bool first = chunk == 0;
  const int32_t* path = a.path + static_cast<long long>(b) * a.N;
  const int most = a.table.max_pages * S;
  const int n = min(max(a.lengths[b], 0), most);
  int bad = n != a.lengths[b] ? kDataLengthRange : 0;
  const int vecs = a.cache.row_bytes() / 16;
  const long long columns = 2ll * a.cache.layers * vecs, column = static_cast<long long>(chunk) * kKeepThreads + tid;
  char* data = nullptr;
  if (column < columns) {
    const int which = static_cast<int>(column / vecs);
    data = (which & 1 ? a.cache.v : a.cache.k) + (which >> 1) * a.cache.layer_stride + (column - static_cast<long long>(which) * vecs) * 16;
  }
  const int base = n - a.N;
  int kept = 0;
  for (int j0 = 0; j0 < a.N; j0 += kKeepMoves) {
    // the path's next entries, up to its end
    if (tid == 0) s_end = min(a.N - j0, kKeepMoves);
    __syncthreads();
    const int j = j0 + tid;
    int from = -1;
    if (tid < kKeepMoves && j < a.N) {
      from = path[j];
      if (from < 0) {
        atomicMin(&s_end, tid);
      } else if (from >= a.N || (j > 0 && from <= path[j - 1])) {
        atomicMin(&s_end, tid);
      }
    }
    __syncthreads();
    const int end = s_end;
    if (tid == end && from >= 0) bad |= kDataPathRange;  // (the entry that ended it)
    if (base < 0) {
      if (end > 0) {
        bad |= kDataLengthRange;
        kept = -1;
      }
      break;
    }
    if (tid < end) {
      s_from[tid] = -1;
      if (from != j) {
        const int t = base + from, d = base + j;
        const int32_t* table = a.table.ids + b * a.table.stride;
        const int page = table[t / S], to = table[d / S];
        if (page < 0 || page >= a.cache.pages || to < 0 || to >= a.cache.pages) {
          bad |= kDataPageRange;
        } else {
          s_from[tid] = page * a.cache.page_stride + t % S * a.cache.token_stride;
          s_to[tid] = to * a.cache.page_stride + d % S * a.cache.token_stride;
        }
      }
    }
    __syncthreads();
    if (data)
      for (int m = 0; m < end; m += 8) {
        uint4 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (m + i < end && s_from[m + i] >= 0) w[i] = *reinterpret_cast<const uint4*>(data + s_from[m + i]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (m + i < end && s_from[m + i] >= 0) *reinterpret_cast<uint4*>(data + s_to[m + i]) = w[i];
      }
    kept += end;
    if (end < kKeepMoves) break;
    __syncthreads();
  }
  if (first) {
    report(a.status, bad);
    if (tid == 0) a.new_lengths[b] = kept < 0 ? n : max(base + kept, 0);
  }
}

}  // namespace

cudaError_t launch_rotated_append(const RotatedAppendArgs& a, int sm_count, cudaStream_t stream) {
  const int esz = a.cache.bf16 ? 2 : 4, kN = 16 / esz, D = a.cache.head_dim;
  const int turned = a.interleaved ? 2 * a.n_freq / kN : a.n_freq / kN, per_head = turned + (D - 2 * a.n_freq) / kN;
  const long long units = static_cast<long long>(a.q_heads + a.cache.heads) * per_head + static_cast<long long>(a.cache.heads) * (D / kN);
  // Warps a token: one wave of the 16 that an SM holds, with a unit a lane at least.  64
  // trees of 16: 16 an SM 8.4 us, 8 and 32 10.3, 64 14.4;  16 trees: 6.2, 6.4, 8.2, 8.2.
  long long parts = static_cast<long long>(sm_count) * 16 / a.T;
  if (parts > (units + 31) / 32) parts = (units + 31) / 32;
  if (parts < 1) parts = 1;
  const long long blocks = (a.T * parts + kAppendWarps - 1) / kAppendWarps;
  const DivU64 by_part = DivU64::make(parts);
  const Div32 by_unit = Div32::make(per_head);
  auto go = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(blocks), kAppendWarps * 32, 0, stream>>>(a, static_cast<int>(parts), by_part, by_unit);
  };
  if (a.cache.bf16) a.interleaved ? go(rotated_append_kernel<BF16, true>) : go(rotated_append_kernel<BF16, false>);
  else a.interleaved ? go(rotated_append_kernel<F32, true>) : go(rotated_append_kernel<F32, false>);
  return cudaGetLastError();
}

cudaError_t launch_tree_accept(const AcceptArgs& a, cudaStream_t stream) {
  tree_accept_kernel<<<(a.B + kAcceptWarps - 1) / kAcceptWarps, kAcceptWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

long long keep_blocks(const CacheView& c) {
  const long long columns = 2ll * c.layers * (c.row_bytes() / 16);
  return (columns + kKeepThreads - 1) / kKeepThreads;
}

cudaError_t launch_keep(const KeepArgs& a, cudaStream_t stream) {
  const long long chunks = keep_blocks(a.cache);
  keep_kernel<<<static_cast<unsigned>(a.B * chunks), kKeepThreads, 0, stream>>>(a, static_cast<unsigned>(chunks));
  return cudaGetLastError();
}

}  // namespace specv
