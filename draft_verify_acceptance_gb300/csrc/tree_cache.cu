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
__device__ __forceinline__ unsigned long long turns_of(float f) {
  constexpr unsigned long long kInv2Pi = 0x28be60db9391054aull;  // 2^64 / (2 pi)
  const uint32_t u = __float_as_uint(f), e = (u >> 23) & 255;
  const unsigned long long m = e ? (u & 0x7fffffu) | 0x800000u : u & 0x7fffffu;
  const unsigned long long lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  const int shift = 150 - static_cast<int>(e ? e : 1);  // |f| = m * 2^-shift
  unsigned long long t;
  if (shift >= 128) t = 0;
  else if (shift >= 64) t = hi >> (shift - 64);
  else if (shift > 0) t = (lo >> shift) | (hi << (64 - shift));
  else t = shift > -64 ? lo << -shift : 0;
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

// A token's work in units: a unit of a rotated head is a piece of 16 bytes and
// the one n_freq dimensions on (interleaved: one piece, its pairs side by side),
// or a piece behind the rotated dimensions; then come the values' pieces.
template <typename E, bool kInterleaved>
__global__ void __launch_bounds__(kAppendWarps * 32)
rotated_append_kernel(const RotatedAppendArgs a, int parts, DivU64 by_part, DivU64 by_unit) {
  constexpr int kN = Piece<E>::kN;
  __shared__ float2 s_turn[kAppendWarps][kMaxFreq];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long job = static_cast<long long>(blockIdx.x) * kAppendWarps + warp;
  const int row = static_cast<int>(by_part(static_cast<unsigned long long>(job)));
  const int part = static_cast<int>(job - static_cast<long long>(row) * parts);
  if (row >= a.T) return;
  const int D = a.cache.head_dim, F = a.n_freq, H = a.cache.heads;

  // the token's sequence and place
  int b, after, bad = 0;
  bool claimed = true;
  if (a.starts) {
    int lo = 0, hi = a.B;  // the last b with starts[b] <= row
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.starts[mid] <= row) lo = mid;
      else hi = mid;
    }
    b = lo;
    after = a.starts[b + 1] - row;
    claimed = a.starts[b] <= row && after > 0 && a.starts[b + 1] <= a.T;
  } else {
    const int per = a.T / a.B;
    b = row / per;
    after = per - (row - b * per);
  }
  long long off = -1;
  int at = 0;
  if (claimed) {
    const long long place = static_cast<long long>(a.lengths[b]) - after;
    at = static_cast<int>(place);
    if (place < 0 || place >= static_cast<long long>(a.table.max_pages) * a.cache.page_size) {
      bad = kDataLengthRange;
    } else {
      const int slot = at / a.cache.page_size;
      const int page = a.table.ids[b * a.table.stride + slot];
      if (page < 0 || page >= a.cache.pages) bad = kDataPageRange;
      else off = page * a.cache.page_stride + (at - slot * a.cache.page_size) * a.cache.token_stride;
    }
  } else {
    bad = kDataLengthRange;
  }
  if (part == 0 && lane == 0) report(a.status, bad);
  const char* q = a.q + row * a.q_stride;
  char* q_out = a.q_out + row * a.q_out_stride;
  if (!claimed) {
    if (a.q_out != a.q)
      for (int j = part * 32 + lane; j < a.q_heads * (D / kN); j += parts * 32)
        reinterpret_cast<uint4*>(q_out)[j] = make_uint4(0, 0, 0, 0);
    return;
  }

  const long long position = a.positions ? a.positions[row] : at;
  for (int i = lane; i < F; i += 32)
    s_turn[warp][i] = cos_sin(static_cast<uint32_t>((static_cast<unsigned long long>(position) * turns_of(a.inv_freq[i])) >> 32));
  __syncwarp();

  const int turned = kInterleaved ? 2 * F / kN : F / kN, per_head = turned + (D - 2 * F) / kN;
  const int rotated = (a.q_heads + (off >= 0 ? H : 0)) * per_head, units = rotated + (off >= 0 ? H * (D / kN) : 0);
  for (int j = part * 32 + lane; j < units; j += parts * 32) {
    if (j >= rotated) {
      const int e = j - rotated;
      reinterpret_cast<uint4*>(a.cache.v + off)[e] = ld_stream_v4(reinterpret_cast<const uint4*>(a.v_new + row * a.new_stride) + e);
      continue;
    }
    const int head = static_cast<int>(by_unit(static_cast<unsigned long long>(j))), u = j - head * per_head;
    const bool is_q = head < a.q_heads;
    const long long in = static_cast<long long>(is_q ? head : head - a.q_heads) * D * E::kBytes;
    const uint4* from = reinterpret_cast<const uint4*>((is_q ? q : a.k_new + row * a.new_stride) + in);
    uint4* to = reinterpret_cast<uint4*>((is_q ? q_out : a.cache.k + off) + in);
    if (u >= turned) {
      const int e = 2 * F / kN + u - turned;
      to[e] = from[e];
    } else if constexpr (kInterleaved) {
      float x[kN];
      Piece<E>::unpack(from[u], x);
#pragma unroll
      for (int i = 0; i < kN; i += 2) {
        const float2 t = s_turn[warp][(u * kN + i) / 2];
        const float p = x[i], r = x[i + 1];
        x[i] = p * t.x - r * t.y;
        x[i + 1] = r * t.x + p * t.y;
      }
      to[u] = Piece<E>::pack(x);
    } else {
      float x[kN], y[kN];
      Piece<E>::unpack(from[u], x);
      Piece<E>::unpack(from[u + turned], y);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float2 t = s_turn[warp][u * kN + i];
        const float p = x[i], r = y[i];
        x[i] = p * t.x - r * t.y;
        y[i] = r * t.x + p * t.y;
      }
      to[u] = Piece<E>::pack(x);
      to[u + turned] = Piece<E>::pack(y);
    }
  }
}

// ---- accept --------------------------------------------------------------------
// One warp a tree, a lane holding nodes lane, lane + 32, ...: a step compares all
// of them with (node, drawn token) and takes the lowest match.
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
// what a store of it has written.
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
    // the path's entries of this round, up to its end
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
  // warps a token: enough to fill the GPU, with a unit a lane at least
  long long parts = static_cast<long long>(sm_count) * 32 / a.T;
  if (parts > (units + 31) / 32) parts = (units + 31) / 32;
  if (parts < 1) parts = 1;
  const long long blocks = (a.T * parts + kAppendWarps - 1) / kAppendWarps;
  const DivU64 by_part = DivU64::make(parts), by_unit = DivU64::make(per_head);
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
