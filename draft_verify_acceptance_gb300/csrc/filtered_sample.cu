// filtered_sample.cu -- sampling from truncated distributions on sm_103a:
// temperature, top-k, min-p, top-p and one draw per row (the definition is in
// include/spec_decode.h).
//
// Weights are integers, w = round(2^40 * 2^t), so sums are exact in any
// order and every cut and draw is the same whatever the schedule: "the first
// element, in the order of a key, at which the running sum of weights passes
// a threshold".  The key is (descending logit, ascending index) for the cuts
// and the index for the draw.
//
// One cluster of C blocks per row, each block's slice of the row in shared
// memory (TMA bulk copies), so the row crosses HBM once.
//   1. As the copies land every thread keeps its largest logit.  The cluster
//      exchanges the row's maximum and a threshold tau: a low order statistic
//      of the threads' maxima, above which a few hundred logits lie.
//   2. One sweep over the slice sums every weight (only when the cuts need the
//      whole row's sum: top-p alone, or no cut at all) and lists the logits
//      from tau up.  What a cut keeps nearly always lies in that list: the k
//      largest, what min-p leaves, the share of the mass that top-p asks for.
//      Whether it does is known exactly from counts and sums.
//   3. The list goes to one block, which makes the cuts and the draw on it:
//      a 256-bin histogram of weights over the key's range, one warp for the
//      at most 32 candidates of the crossing bin.
// A row without cuts draws from the sweep's sums by 32-vector group.  A row
// whose kept set does not lie in the list (flat distributions, a large k)
// takes the same cuts by histograms over the slices, level by level.
#include <cooperative_groups.h>

#include <cfloat>
#include <climits>

#include "device_common.cuh"
#include "launch_decode.h"
#include "sample_common.cuh"

namespace cg = cooperative_groups;

namespace specv {
namespace {

constexpr int kThreadsS = 512;
constexpr int kWarpsS = kThreadsS / 32;
constexpr int kMaxCS = 8;               // blocks of a cluster
constexpr int kDepth = 12;              // listed logits a thread holds
constexpr int kList = 1024;             // listed logits of a row
constexpr int kPerThread = kList / kThreadsS;
constexpr int kGroups = kList / kWarpsS;  // rounds with group sums of their own (they share the list's memory)
constexpr long long kSliceBytesS = 65024;     // a slice, while more blocks can share the row
constexpr long long kMaxSliceS = 128 * 1024;  // a slice of the largest cluster (65536 bf16: 16-bit places)
constexpr int kChunkS = 1024;           // vectors per bulk copy
constexpr int kMaxChunksS = 8;
static_assert(kMaxSliceS / 16 <= kChunkS * kMaxChunksS, "bulk copies of a slice");

// 2^f on [-1/2, 1/2] times 2^40: 1 + f (c1 + f (c2 + ...)), a minimax fit of
// the relative error (9.2e-8; 1.9e-7 with the roundings of every operation).
// The factor 2^40 is exact and changes no rounding.
constexpr float kScale = 1099511627776.f;
constexpr float kC1 = 0.6931470036506653f, kC2 = 0.24022242426872253f, kC3 = 0.05550733581185341f,
                kC4 = 0.009671513922512531f, kC5 = 0.0013264728477224708f;
constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number

// The weight of a logit x of a row with largest logit M and scale s = log2(e) / T.
__device__ __forceinline__ unsigned long long weight(float x, float M, float s) {
  const float t = fmaxf(__fmul_rn(__fsub_rn(x, M), s), -64.f);
  const float r = __fadd_rn(t, kRound);
  const float f = __fsub_rn(t, __fsub_rn(r, kRound));
  float g = kC5 * kScale;
  g = __fadd_rn(__fmul_rn(g, f), kC4 * kScale);
  g = __fadd_rn(__fmul_rn(g, f), kC3 * kScale);
  g = __fadd_rn(__fmul_rn(g, f), kC2 * kScale);
  g = __fadd_rn(__fmul_rn(g, f), kC1 * kScale);
  g = __fadd_rn(__fmul_rn(g, f), kScale);
  // times 2^n: n sits in the low bits of r
  return __float2ull_rn(__uint_as_float(__float_as_uint(g) + (__float_as_uint(r) << 23)));
}

// Bits that order floats from largest to smallest (+0 and -0 alike).
__device__ __forceinline__ unsigned int falling(float x) {
  const unsigned int b = __float_as_uint(x + 0.f);
  return ~((b >> 31) ? ~b : (b | 0x80000000u));
}

// A row's settings.
struct Settings {
  float T, top_p, min_p;
  int k;  // V: off
  int bad;
};
__device__ __forceinline__ Settings settings_of(const SampleArgs& a, int row) {
  Settings s;
  s.bad = 0;
  s.T = a.temperatures ? a.temperatures[row] : a.temperature;
  s.k = a.top_ks ? a.top_ks[row] : a.top_k;
  s.top_p = a.top_ps ? a.top_ps[row] : a.top_p;
  s.min_p = a.min_ps ? a.min_ps[row] : a.min_p;
  if (s.k <= 0 || s.k > a.V) s.k = a.V;
  if (!(s.T >= 0.f && s.T < INFINITY)) {
    s.T = 1.f;
    s.bad = kDataParamRange;
  }
  if (isnan(s.top_p)) {
    s.top_p = 1.f;
    s.bad = kDataParamRange;
  }
  if (isnan(s.min_p)) {
    s.min_p = 0.f;
    s.bad = kDataParamRange;
  }
  if (s.T < 7.9e-31f) {  // 0, or so small that log2(e) / T could overflow
    s.T = 1.f;
    s.k = 1;
  }
  return s;
}

// The fast sweep's sum: the two weights of a pair of logits, in packed fp32
// arithmetic with the same roundings, added to sums of their parts.  With y
// = 2^40 2^t as a float, high = y rounded to a multiple of 2^20 and low =
// round(y - high) are read off the mantissas of y + 1.5 * 2^43 and (y -
// high) + 1.5 * 2^23; high is even, so high + low is round(y).
struct Sum {
  unsigned int high = 0, low = 0;  // with the constants' bits still in
};
constexpr float kHigh = 13194139533312.f;  // 1.5 * 2^43

// A product rounded by itself.  A packed multiplication that feeds a packed
// addition is fused by the assembler although both name their rounding (one
// weight in eight then differed), so the product is a fused multiply-add of
// a -0 that only the launch knows.
__device__ __forceinline__ float2 fmul2(float2 a, float2 b, float minus_zero) {
  return ffma2(a, b, make_float2(minus_zero, minus_zero));
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ float2 add_pair(Sum& z, float2 x, float M, float s, float mz) {
  float2 t = fmul2(fadd2(x, both(-M)), both(s), mz);
  t.x = fmaxf(t.x, -64.f);
  t.y = fmaxf(t.y, -64.f);
  const float2 r = fadd2(t, both(kRound));
  const float2 n = fadd2(r, both(-kRound));
  const float2 f = fadd2(t, make_float2(-n.x, -n.y));
  float2 g = both(kC5 * kScale);
  g = fadd2(fmul2(g, f, mz), both(kC4 * kScale));
  g = fadd2(fmul2(g, f, mz), both(kC3 * kScale));
  g = fadd2(fmul2(g, f, mz), both(kC2 * kScale));
  g = fadd2(fmul2(g, f, mz), both(kC1 * kScale));
  g = fadd2(fmul2(g, f, mz), both(kScale));
  float2 y;
  y.x = __uint_as_float(__float_as_uint(g.x) + (__float_as_uint(r.x) << 23));
  y.y = __uint_as_float(__float_as_uint(g.y) + (__float_as_uint(r.y) << 23));
  const float2 h = fadd2(y, both(kHigh));
  const float2 e = fadd2(h, both(-kHigh));
  const float2 l = fadd2(fadd2(y, make_float2(-e.x, -e.y)), both(kRound));
  z.high += __float_as_uint(h.x) + __float_as_uint(h.y);
  z.low += __float_as_uint(l.x) + __float_as_uint(l.y);
  return y;  // a weight is 0 up to y = 1/2
}
// The whole number behind the sums of n weights.
__device__ __forceinline__ unsigned long long value_of(const Sum& z, unsigned int n) {
  const unsigned int high = z.high - n * __float_as_uint(kHigh);
  const int low = static_cast<int>(z.low - n * __float_as_uint(kRound));
  return (static_cast<unsigned long long>(high) << 20) + static_cast<long long>(low);
}

// Which tokens are kept: key (falling(x), index) at most `cut`, weight at
// least `least` (weight 0 is never kept).
struct Kept {
  unsigned long long cut, least;
};
__device__ __forceinline__ unsigned long long cut_key(float x, unsigned int j) {
  return (static_cast<unsigned long long>(falling(x)) << 22) | j;
}

// -inf as an element.
template <typename E>
__device__ __forceinline__ typename E::raw masked_value() {
  if constexpr (E::kBytes == 2) return 0xff80;
  else return -INFINITY;
}

// A block's slice of a row: vectors [0, nv) of 16 bytes, in shared memory or
// (rows too long for a cluster) read from global memory each time.  Vectors
// past the row's end are filled with -inf.
template <typename E, bool kStaged>
struct Slice {
  const uint4* staged;
  const typename E::raw* global;
  int nv, first, V;  // vectors; index of the first element; elements of the row
  int width;         // 32-vector steps a warp takes per round
  __device__ __forceinline__ uint4 at(int v) const {
    if constexpr (kStaged) {
      return staged[v];
    } else {
      constexpr int kVec = Staged<E>::kVec;
      typename E::raw x[kVec];
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        const int j = v * kVec + k;
        x[k] = first + j < V ? __ldg(global + j) : masked_value<E>();
      }
      uint4 w;
      memcpy(&w, x, 16);
      return w;
    }
  }
  // Round c, step i: the vector of this thread.  A warp's vectors of a round
  // are contiguous, rounds follow each other.
  __device__ __forceinline__ int vec(int c, int i) const {
    return ((c * kWarpsS + (threadIdx.x >> 5)) * width + i) * 32 + (threadIdx.x & 31);
  }
  __device__ __forceinline__ int rounds() const {
    return (nv + kThreadsS * width - 1) / (kThreadsS * width);
  }
};

template <typename E>
__device__ __forceinline__ float element(const uint4& w, int k) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  if constexpr (E::kBytes == 4) return __uint_as_float(u[k]);
  return (k & 1) ? bf16_hi(u[k >> 1]) : bf16_lo(u[k >> 1]);
}

// A running maximum of 16-byte vectors that keeps a NaN.
template <typename E>
struct Peak;
template <>
struct Peak<BF16> {
  uint32_t m = 0xff80ff80u;  // (-inf, -inf)
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  __device__ __forceinline__ void take(const uint4& w) { m = max2(m, max2(max2(w.x, w.y), max2(w.z, w.w))); }
  __device__ __forceinline__ float value() const {
    const uint32_t x = max2(m, __byte_perm(m, 0, 0x1032));
    return bf16_lo(x);
  }
};
template <>
struct Peak<F32> {
  float m = -INFINITY;
  static __device__ __forceinline__ float max2(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
  }
  __device__ __forceinline__ void take(const uint4& w) {
    m = max2(m, max2(max2(__uint_as_float(w.x), __uint_as_float(w.y)), max2(__uint_as_float(w.z), __uint_as_float(w.w))));
  }
  __device__ __forceinline__ float value() const { return m; }
};

// Which elements of a vector are at least `from`: bit k for element k.
template <typename E>
__device__ __forceinline__ uint32_t at_least(const uint4& w, float from) {
  uint32_t hit = 0;
#pragma unroll
  for (int k = 0; k < Staged<E>::kVec; ++k) hit |= (element<E>(w, k) >= from ? 1u : 0u) << k;
  return hit;
}

// The logit of a cut key; the lowest finite one for "no cut".
__device__ __forceinline__ float logit_of(unsigned long long cut) {
  if (cut == ~0ull) return -FLT_MAX;
  const unsigned int o = ~static_cast<unsigned int>(cut >> 22);
  return __uint_as_float((o >> 31) ? o & 0x7fffffffu : ~o);
}

// What every rank of a cluster publishes to all.
struct Exchange {
  float max[kMaxCS], tau[kMaxCS];  // tau: sum of the warps' order statistics, taus of them
  int taus[kMaxCS], listed[kMaxCS];                         // listed: -1 when a thread's list overflowed
  unsigned long long sum[kMaxCS], listed_sum[kMaxCS];
  unsigned long long mass[kMaxCS], count[kMaxCS];
};

struct Shared {
  Exchange x;
  unsigned long long part[kWarpsS], part2[kWarpsS];
  float wmax[kWarpsS], wtau[kWarpsS];
  unsigned long long few_key[32], few_w[32];
  unsigned long long rem, lo, cut;
  unsigned int n_few, bin_count;
  unsigned int list_n;
  int scan[kWarpsS];
  int sel[4];
};

// 256 bins of weights, kept as 32-bit parts so that shared memory adds them
// without a loop, and of counts.
struct Bins {
  unsigned int part[4][256], count[256];
  unsigned long long sum[256];  // of the cluster
  unsigned int all[256];
};
template <int kParts>  // parts of 20 bits (a list) or of 11 (a slice)
__device__ __forceinline__ void bin_add(Bins* h, unsigned int at, unsigned long long w) {
  constexpr int kBits = kParts == 2 ? 20 : 11;
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    const unsigned int x = static_cast<unsigned int>(w >> (i * kBits)) & (i == kParts - 1 ? ~0u : (1u << kBits) - 1u);
    if (x) atomicAdd(&h->part[i][at], x);
  }
  atomicAdd(&h->count[at], 1u);
}
template <int kParts>
__device__ __forceinline__ unsigned long long bin_value(const Bins* h, unsigned int at) {
  constexpr int kBits = kParts == 2 ? 20 : 11;
  unsigned long long v = 0;
#pragma unroll
  for (int i = 0; i < kParts; ++i) v += static_cast<unsigned long long>(h->part[i][at]) << (i * kBits);
  return v;
}

struct Ctx {
  Shared* sh;
  Bins* bins;
  int C, rank;
  __device__ __forceinline__ void sync() const {
    if (C == 1) {
      __syncthreads();
    } else {
      __syncwarp();  // the cluster barrier takes whole warps
      cg::this_cluster().sync();
    }
  }
  template <typename T>
  __device__ __forceinline__ T* at(T* p, int r) const {
    return C == 1 ? p : cg::this_cluster().map_shared_rank(p, r);
  }
  __device__ __forceinline__ void clear() const {
    unsigned int* x = &bins->part[0][0];
    for (int i = threadIdx.x; i < 5 * 256; i += kThreadsS) x[i] = 0;
    if (threadIdx.x == 0) sh->n_few = 0;
  }
};

__device__ __forceinline__ unsigned long long block_sum(unsigned long long v, unsigned long long* part) {
  v = warp_sum_u64(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  unsigned long long t = 0;
#pragma unroll
  for (int w = 0; w < kWarpsS; ++w) t += part[w];
  return t;
}

// Two sums at once.
__device__ __forceinline__ void block_sum2(unsigned long long a, unsigned long long b, Shared& sh,
                                           unsigned long long* sa, unsigned long long* sb) {
  a = warp_sum_u64(a);
  b = warp_sum_u64(b);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    sh.part[threadIdx.x >> 5] = a;
    sh.part2[threadIdx.x >> 5] = b;
  }
  __syncthreads();
  *sa = *sb = 0;
#pragma unroll
  for (int w = 0; w < kWarpsS; ++w) {
    *sa += sh.part[w];
    *sb += sh.part2[w];
  }
}

// One warp: the first of 256 bins (by the running sum of value(bin)) to pass
// rem.  Leaves the bin, what is left of rem inside it and its count in `sh`.
template <typename F>
__device__ __forceinline__ void crossing_bin(const Ctx& c, unsigned long long rem, F value) {
  const int lane = threadIdx.x & 31;
  unsigned long long h[8], mine = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] = value(lane * 8 + i);
    mine += h[i];
  }
  unsigned long long before = warp_scan_u64(mine, lane) - mine;
  const unsigned int hit = __ballot_sync(0xffffffffu, before + mine > rem);
  const int owner = hit ? __ffs(hit) - 1 : 31;
  if (lane == owner) {
    int b = 0;
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (b == i && before + h[i] <= rem) {
        before += h[i];
        b = i + 1;
      }
    c.sh->sel[0] = lane * 8 + b;
    c.sh->rem = rem >= before ? rem - before : 0;
    c.sh->bin_count = c.bins->count[lane * 8 + b];
  }
}

// One warp: of at most 32 (key, weight) pairs the lowest key at which the
// running sum in key order passes rem.
__device__ __forceinline__ unsigned long long crossing_of_few(const unsigned long long* keys,
                                                              const unsigned long long* ws, int n,
                                                              unsigned long long rem) {
  const int lane = threadIdx.x & 31;
  const unsigned long long key = lane < n ? keys[lane] : ~0ull, w = lane < n ? ws[lane] : 0ull;
  unsigned long long run = 0;
  for (int i = 0; i < n; ++i) {
    const unsigned long long k2 = __shfl_sync(0xffffffffu, key, i), w2 = __shfl_sync(0xffffffffu, w, i);
    if (k2 <= key) run += w2;
  }
  unsigned long long best = lane < n && run > rem ? key : ~0ull;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
  return best;
}

__device__ __forceinline__ int bin_shift(unsigned long long span) {
  const int bits = 64 - __clzll(static_cast<long long>(span));
  return bits > 8 ? bits - 8 : 0;
}

// The crossing key over the listed elements, which the block's threads hold
// (key, and weight 0 for those outside the set).  Keys lie in [lo, hi].
// kCount: every weight is 1.
template <bool kCount>
__device__ unsigned long long list_crossing(const Ctx& c, const unsigned long long (&key)[kPerThread],
                                            const unsigned long long (&w)[kPerThread], unsigned long long lo,
                                            unsigned long long hi, unsigned long long rem) {
  int shift = bin_shift(hi - lo);
  for (;;) {
    __syncthreads();
    c.clear();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const unsigned long long at = (key[i] - lo) >> shift;
      if (w[i] && key[i] >= lo && at < 256) {
        if (kCount) atomicAdd(&c.bins->count[at], 1u);
        else bin_add<2>(c.bins, static_cast<unsigned int>(at), w[i]);
      }
    }
    __syncthreads();
    if (threadIdx.x < 32)
      crossing_bin(c, rem, [&](int b) -> unsigned long long {
        return kCount ? c.bins->count[b] : bin_value<2>(c.bins, b);
      });
    __syncthreads();
    rem = c.sh->rem;
    lo += static_cast<unsigned long long>(c.sh->sel[0]) << shift;
    if (shift == 0) return lo;
    if (c.sh->bin_count <= 32) break;
    shift = shift > 8 ? shift - 8 : 0;
  }
#pragma unroll
  for (int i = 0; i < kPerThread; ++i)
    if (w[i] && key[i] >= lo && (key[i] - lo) >> shift == 0) {
      const unsigned int at = atomicAdd(&c.sh->n_few, 1u);
      if (at < 32) {
        c.sh->few_key[at] = key[i];
        c.sh->few_w[at] = w[i];
      }
    }
  __syncthreads();
  if (threadIdx.x < 32) {
    const unsigned long long k = crossing_of_few(c.sh->few_key, c.sh->few_w, min(32u, c.sh->n_few), rem);
    if (threadIdx.x == 0) c.sh->lo = k;
  }
  __syncthreads();
  return c.sh->lo;
}

// The crossing cut key over the cluster's slices, for rows whose kept set
// does not lie in the list; measure(index, x) is an element's weight.  The
// first bins are sixths of t, which spreads a row's elements over them; the
// following ones divide the crossing bin's keys.  Every rank gets the key.
template <typename E, bool kStaged, bool kCount, typename F>
__device__ unsigned long long slice_crossing(const Ctx& c, const Slice<E, kStaged>& sl, float M, float s,
                                             unsigned long long rem, F measure) {
  constexpr int VEC = Staged<E>::kVec;
  auto bin_of = [&](float x) { return min(255, static_cast<int>(fmaxf((x - M) * s, -64.f) * -6.f)); };
  // use(index, x) of every element in [from, to]
  auto sweep = [&](float from, float to, auto use) {
    for (int r = 0; r < sl.rounds(); ++r)
      for (int i = 0; i < sl.width; ++i) {
        const int v = sl.vec(r, i);
        if (v >= sl.nv) continue;
        const uint4 w = sl.at(v);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float x = element<E>(w, k);
          if (x >= from && x <= to) use(sl.first + v * VEC + k, x);
        }
      }
  };
  int shift = -1, bin = 0;  // -1: bins of t
  unsigned long long lo = 0;
  float from = -INFINITY, to = INFINITY;
  for (;;) {
    c.sync();  // what other ranks read is free
    c.clear();
    __syncthreads();
    sweep(from, to, [&](unsigned int j, float x) {
      unsigned int at = bin_of(x);
      if (shift >= 0) {
        const unsigned long long key = cut_key(x, j), d = (key - lo) >> shift;
        if (static_cast<int>(at) != bin || key < lo || d > 255) return;
        at = static_cast<unsigned int>(d);
      }
      if (kCount) {
        atomicAdd(&c.bins->count[at], 1u);
      } else {
        const unsigned long long w = measure(j, x);
        if (w) bin_add<4>(c.bins, at, w);
      }
    });
    c.sync();
    if (threadIdx.x < 256) {
      unsigned long long w = 0;
      unsigned int n = 0;
      for (int r = 0; r < c.C; ++r) {
        const Bins* h = c.at(c.bins, r);
        n += h->count[threadIdx.x];
        if (!kCount) w += bin_value<4>(h, threadIdx.x);
      }
      c.bins->sum[threadIdx.x] = kCount ? n : w;
      c.bins->all[threadIdx.x] = n;
    }
    __syncthreads();
    if (threadIdx.x < 32) crossing_bin(c, rem, [&](int b) { return c.bins->sum[b]; });
    __syncthreads();
    rem = c.sh->rem;
    const int b = c.sh->sel[0];
    const bool few = c.bins->all[b] <= 32;
    if (shift < 0) {
      // the bin's logits, with room for the roundings of t and of these bounds
      bin = b;
      const float unit = __fdiv_rn(1.f, 6.f * s);
      to = fminf(M, M - (b - 0.01f) * unit);
      to = fminf(M, to + fabsf(to) * 4.8e-7f);
      from = b == 255 ? -INFINITY : M - (b + 1.01f) * unit;
      from -= b == 255 ? 0.f : fabsf(from) * 4.8e-7f;
      lo = cut_key(to, 0);
      shift = bin_shift(cut_key(from, 0x3fffff) - lo);
      if (few) {
        shift = 54;  // all keys of the bin at once
        break;
      }
      continue;
    }
    lo += static_cast<unsigned long long>(b) << shift;
    if (shift == 0) return lo;
    if (few) break;
    shift = shift > 8 ? shift - 8 : 0;
  }
  Shared* zero = c.at(c.sh, 0);
  sweep(from, to, [&](unsigned int j, float x) {
    const unsigned long long key = cut_key(x, j);
    if (bin_of(x) == bin && key >= lo && (key - lo) >> shift == 0) {
      const unsigned long long w = kCount ? 1ull : measure(j, x);
      if (w) {
        const unsigned int at = atomicAdd(&zero->n_few, 1u);
        if (at < 32) {
          zero->few_key[at] = key;
          zero->few_w[at] = w;
        }
      }
    }
  });
  c.sync();
  if (threadIdx.x < 32) {
    const unsigned long long k = crossing_of_few(zero->few_key, zero->few_w, min(32u, zero->n_few), rem);
    if (threadIdx.x == 0) c.sh->lo = k;
  }
  c.sync();
  return c.sh->lo;
}

// Sums of the kept weights by group (a warp's vectors of a round), the
// cluster's total and count in the exchange.
template <typename E, bool kStaged, typename F>
__device__ void group_sums(const Ctx& c, const Slice<E, kStaged>& sl, unsigned long long* groups, F vector_sum,
                           unsigned long long* S, unsigned long long* count) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long mine = 0, n = 0;
  for (int r = 0; r < sl.rounds(); ++r) {
    unsigned long long g = 0;
    for (int i = 0; i < sl.width; ++i) {
      const int v = sl.vec(r, i);
      if (v < sl.nv) {
        unsigned int k = 0;
        g += vector_sum(v, &k);
        n += k;
      }
    }
    mine += g;
    g = warp_sum_u64(g);
    if (lane == 0) groups[r * kWarpsS + warp] = g;
  }
  unsigned long long t, k;
  block_sum2(mine, n, *c.sh, &t, &k);
  if (threadIdx.x < c.C) {
    *c.at(&c.sh->x.mass[c.rank], threadIdx.x) = t;
    *c.at(&c.sh->x.count[c.rank], threadIdx.x) = k;
  }
  c.sync();
  *S = *count = 0;
  for (int r = 0; r < c.C; ++r) {
    *S += c.sh->x.mass[r];
    *count += c.sh->x.count[r];
  }
}

// The draw from group sums: the rank that holds the crossing returns the
// token, the others -1.  element_weight(index, x) as in group_sums.
template <typename E, bool kStaged, typename F>
__device__ int group_draw(const Ctx& c, const Slice<E, kStaged>& sl, const unsigned long long* groups,
                          unsigned long long theta, F element_weight) {
  constexpr int VEC = Staged<E>::kVec;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int owner = c.C - 1;
  unsigned long long off = 0;
  for (int r = 0; r < c.C; ++r) {
    if (off + c.sh->x.mass[r] > theta) {
      owner = r;
      break;
    }
    off += c.sh->x.mass[r];
  }
  if (c.rank != owner) return -1;
  if (warp == 0) {
    unsigned long long rem = theta - min(off, theta);
    // the group: 32 at a time
    const int n = sl.rounds() * kWarpsS;
    int group = -1;
    for (int g0 = 0; g0 < n && group < 0; g0 += 32) {
      const unsigned long long m = g0 + lane < n ? groups[g0 + lane] : 0ull;
      const unsigned long long incl = warp_scan_u64(m, lane);
      const unsigned int hit = __ballot_sync(0xffffffffu, incl > rem);
      if (hit) {
        const int at = __ffs(hit) - 1;
        group = g0 + at;
        rem -= __shfl_sync(0xffffffffu, incl - m, at);
      } else {
        rem -= __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    int token = sl.first;  // (only a timed-out load leaves no crossing)
    // the vector in the group, the element in the vector
    for (int i = 0; i < sl.width && group >= 0; ++i) {
      const int v = (group * sl.width + i) * 32 + lane;
      unsigned long long e[VEC], m = 0;
#pragma unroll
      for (int k = 0; k < VEC; ++k) e[k] = 0;
      if (v < sl.nv) {
        const uint4 w = sl.at(v);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          e[k] = element_weight(sl.first + v * VEC + k, element<E>(w, k));
          m += e[k];
        }
      }
      const unsigned long long incl = warp_scan_u64(m, lane);
      const unsigned int hit = __ballot_sync(0xffffffffu, incl > rem);
      if (hit) {
        const int at = __ffs(hit) - 1;
        if (lane == at) {
          unsigned long long left = rem - (incl - m);
          int k = 0;
#pragma unroll
          for (int q = 0; q < VEC - 1; ++q)
            if (k == q && e[q] <= left) {
              left -= e[q];
              k = q + 1;
            }
          token = sl.first + v * VEC + k;
        }
        token = __shfl_sync(0xffffffffu, token, at);
        break;
      }
      rem -= __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) c.sh->sel[1] = token;
  }
  __syncthreads();
  return c.sh->sel[1];
}

// Ascending bitonic sort of one float a lane.
__device__ __forceinline__ float warp_sort(float x, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, x, j);
      const bool up = (lane & k) == 0 || k == 32, low = (lane & j) == 0;
      x = (up == low) ? fminf(x, y) : fmaxf(x, y);
    }
  return x;
}

// How many logits the list should hold, and which of a warp's 32 sorted
// maxima says so: with m logits listed among T threads a thread holds none
// with probability e^(-m/T), so the threshold is that quantile of the
// maxima.  Averaged over the row's warps it lists m within a tenth on normal
// rows, up to 1.5 m on Zipf-shifted ones (counted).
__device__ __forceinline__ int tau_lane(const Settings& set, int V, int C) {
  const float m = set.k < V ? fminf(1.25f * set.k + 64.f, 700.f) : 640.f;
  const float below = ex2(-1.44269504f * m / (kThreadsS * C));
  return min(31, max(0, static_cast<int>(32.f * below)));
}

// A vector of the filtered row.  Most elements fail the comparison with the
// cut's logit; the others are tested exactly.
template <typename E>
__device__ __forceinline__ void write_kept(const SampleArgs& a, int row, int first, int v, const uint4& w,
                                           bool vectors, const Kept& kept, float edge, float M, float s) {
  constexpr int VEC = Staged<E>::kVec;
  using raw = typename E::raw;
  raw x[VEC];
  memcpy(x, &w, 16);
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    const float f = element<E>(w, k);
    bool in = f >= edge;
    if (in) in = cut_key(f, first + v * VEC + k) <= kept.cut && weight(f, M, s) >= kept.least;
    if (!in) x[k] = masked_value<E>();
  }
  raw* dst = static_cast<raw*>(a.filtered) + static_cast<size_t>(row) * a.V + first + v * VEC;
  if (vectors) {
    uint4 o;
    memcpy(&o, x, 16);
    *reinterpret_cast<uint4*>(dst) = o;
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      if (first + v * VEC + k < a.V) dst[k] = x[k];
  }
}

template <typename E, bool kStaged>
__global__ void __launch_bounds__(kThreadsS, 2)
filtered_sample_kernel(const SampleArgs a, int nvec, int nvs, bool aligned_in, bool aligned_out, float mz) {
  constexpr int VEC = Staged<E>::kVec;
  using raw = typename E::raw;
  extern __shared__ __align__(128) uint4 dyn[];  // slice [nvs] | list [kList] | threads' lists, later the bins
  __shared__ Shared sh;
  __shared__ __align__(8) unsigned long long bars[kMaxChunksS];
  cg::cluster_group cluster = cg::this_cluster();
  Ctx c;
  c.sh = &sh;
  c.C = static_cast<int>(cluster.num_blocks());
  c.rank = static_cast<int>(cluster.block_rank());
  uint4* slice = dyn;
  uint2* list = reinterpret_cast<uint2*>(dyn + (kStaged ? nvs : 0));          // (x, index)
  unsigned long long* groups = reinterpret_cast<unsigned long long*>(list);   // shares the list's memory
  uint16_t* deep = reinterpret_cast<uint16_t*>(list + kList);                 // [kDepth][threads]
  c.bins = reinterpret_cast<Bins*>(list + kList);                             // shares it
  const int lgC = __ffs(c.C) - 1;
  const int row = static_cast<int>(blockIdx.x >> lgC);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int v0 = static_cast<int>((static_cast<long long>(nvec) * c.rank) >> lgC);
  Slice<E, kStaged> sl;
  sl.nv = static_cast<int>((static_cast<long long>(nvec) * (c.rank + 1)) >> lgC) - v0;
  sl.first = v0 * VEC;
  sl.V = a.V;
  sl.staged = slice;
  sl.global = static_cast<const raw*>(a.logits) + row * a.row_stride + sl.first;
  sl.width = kStaged ? 1 : (sl.nv + kThreadsS * kGroups - 1) / (kThreadsS * kGroups);
  if (!kStaged && sl.width < 1) sl.width = 1;

  // ---- the slice into shared memory -------------------------------------
  const int nch = (sl.nv + kChunkS - 1) / kChunkS;
  const bool bulk = kStaged && aligned_in;
  if (bulk) {
    if (tid == 0) {
      for (int k = 0; k < nch; ++k) mbar_init(&bars[k], 1);
      fence_barrier_init();
      for (int k = 0; k < nch; ++k) {
        const uint32_t bytes = min(kChunkS, sl.nv - k * kChunkS) * 16u;
        mbar_arrive_expect_tx(&bars[k], bytes);
        bulk_load(slice + k * kChunkS, sl.global + static_cast<size_t>(k) * kChunkS * VEC, bytes, &bars[k]);
      }
    }
  } else if (kStaged) {  // rows that are not 16-byte aligned: element by element
    raw* dst = reinterpret_cast<raw*>(slice);
    for (int j = tid; j < sl.nv * VEC; j += kThreadsS)
      dst[j] = sl.first + j < a.V ? __ldg(sl.global + j) : masked_value<E>();
  }
  if (tid == 0) {
    sh.list_n = 0;
    sh.n_few = 0;
  }
  const Settings set = settings_of(a, row);
  const float u = a.uniforms[row];
  const float s = __fdiv_rn(1.44269502f, set.T);
  __syncthreads();
  if (c.C > 1) cluster_arrive_relaxed();  // matched before the first store to another block

  // ---- 1. the row's maximum and the list's threshold ----------------------
  bool landed = true;
  Peak<E> peak;
  if (bulk) {
    for (int k = 0; k < nch; ++k) {
      if (!mbar_wait_sleep(&bars[k], 0u)) {
        landed = false;
        break;
      }
      const int stop = min((k + 1) * kChunkS, sl.nv);
#pragma unroll 2
      for (int v = k * kChunkS + tid; v < stop; v += kThreadsS) peak.take(slice[v]);
    }
  } else {
    for (int v = tid; v < sl.nv; v += kThreadsS) peak.take(sl.at(v));
  }
  const float mine = peak.value();
  const bool odd = __any_sync(0xffffffffu, isnan(mine));
  const float sorted = warp_sort(mine, lane);
  const float order = __shfl_sync(0xffffffffu, sorted, tau_lane(set, a.V, c.C));
  if (lane == 31) {
    sh.wmax[warp] = odd ? INFINITY : sorted;
    sh.wtau[warp] = order;
  }
  const int timeout = __syncthreads_or(!landed);
  if (c.C > 1) cluster_wait();  // every block of the cluster has started
  if (tid < c.C) {
    float m = -INFINITY, t = 0.f;
    int n = 0;
#pragma unroll
    for (int w = 0; w < kWarpsS; ++w) {
      m = fmaxf(m, sh.wmax[w]);
      if (sh.wtau[w] > -INFINITY) {
        t += sh.wtau[w];
        ++n;
      }
    }
    *c.at(&sh.x.max[c.rank], tid) = m;
    *c.at(&sh.x.tau[c.rank], tid) = t;
    *c.at(&sh.x.taus[c.rank], tid) = n;
  }
  c.sync();
  float M = -INFINITY, tau = 0.f;
  int taus = 0;
  for (int r = 0; r < c.C; ++r) {
    M = fmaxf(M, sh.x.max[r]);
    tau += sh.x.tau[r];
    taus += sh.x.taus[r];
  }
  tau = taus ? fminf(tau / taus, M) : -INFINITY;
  M += 0.f;
  const bool good = M > -INFINITY && M < INFINITY;
  Kept kept;
  kept.cut = ~0ull;
  kept.least = max(1ull, __float2ull_rn(__fmul_rn(fminf(fmaxf(set.min_p, 0.f), 1.f), kScale)));
  const bool has_k = set.k < a.V, has_m = set.min_p > 0.f, has_p = set.top_p < 1.f;
  const float p_clamped = fminf(fmaxf(set.top_p, 0.f), 0.99999994f);
  unsigned long long S = 0, count = 0;
  int token = -1;  // on the rank that finds it

  float edge = -FLT_MAX;  // the cut's logit
  auto weigh = [&](unsigned int j, float x) -> unsigned long long {
    if (!(x >= edge) || cut_key(x, j) > kept.cut) return 0ull;
    const unsigned long long w = weight(x, M, s);
    return w >= kept.least ? w : 0ull;
  };

  if (good) {
    bool covered = false;
    if (has_k || has_m || has_p) {
      // ---- 2. sum and list ----
      // below `floor` every weight is 0
      const float floor = M - __fdiv_rn(42.f, s);
      const bool complete = !(tau > floor);
      const float from = complete ? floor : tau;
      const bool whole = !has_k && !has_m;  // top-p of the whole row's mass
      Sum z;
      int n = 0;
      unsigned int vectors = 0;
      auto put = [&](const uint4& w, int v) {
        for (uint32_t hit = at_least<E>(w, from); hit; hit &= hit - 1) {
          if (n < kDepth) deep[n * kThreadsS + tid] = static_cast<uint16_t>(v * VEC + __ffs(hit) - 1);
          ++n;
        }
      };
      const bool lists = kStaged && !timeout;
      if (lists) {
        if (whole) {
          for (int v = tid; v < sl.nv; v += kThreadsS) {
            const uint4 w = slice[v];
            float2 x[VEC / 2];
            unpack_pairs<E>(w, x);
#pragma unroll
            for (int k = 0; k < VEC / 2; ++k) add_pair(z, x[k], M, s, mz);
            ++vectors;
            put(w, v);
          }
        } else {
          for (int v = tid; v < sl.nv; v += kThreadsS) put(slice[v], v);
        }
      }
      // the listed weights' sum, and the list to rank 0
      int incl = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
      }
      if (lane == 31) sh.scan[warp] = incl;
      const int over = __syncthreads_or(n > kDepth || !lists);
      int before = incl - n, all = 0;
#pragma unroll
      for (int w = 0; w < kWarpsS; ++w) {
        if (w < warp) before += sh.scan[w];
        all += sh.scan[w];
      }
      if (tid == 0) sh.sel[2] = over ? 0 : static_cast<int>(atomicAdd(c.at(&sh.list_n, 0), static_cast<unsigned int>(all)));
      __syncthreads();
      const int base = sh.sel[2];
      unsigned long long lw = 0;
      if (!over) {
        uint2* to = c.at(list, 0);
        for (int i = 0; i < n; ++i) {
          const int e = deep[i * kThreadsS + tid];
          const float x = staged_elem<E>(slice, e);
          if (whole) lw += weight(x, M, s);  // the sum decides whether the list covers top-p
          if (base + before + i < kList)
            to[base + before + i] = make_uint2(__float_as_uint(x), static_cast<unsigned int>(sl.first + e));
        }
      }
      unsigned long long zs = 0;
      if (whole) block_sum2(value_of(z, vectors * VEC), lw, sh, &zs, &lw);
      if (tid < c.C) {
        *c.at(&sh.x.sum[c.rank], tid) = zs;
        *c.at(&sh.x.listed_sum[c.rank], tid) = lw;
        *c.at(&sh.x.listed[c.rank], tid) = over ? -1 : all;
      }
      c.sync();
      int listed = 0;
      bool overflow = false;
      unsigned long long Z = 0, L = 0;
      for (int r = 0; r < c.C; ++r) {
        overflow |= sh.x.listed[r] < 0;
        listed += sh.x.listed[r];
        Z += sh.x.sum[r];
        L += sh.x.listed_sum[r];
      }
      overflow |= listed > kList;
      // does the list hold all that can be kept?
      if (!overflow) {
        if (complete) {
          covered = true;
        } else if (has_k) {
          covered = listed >= set.k;
        } else if (has_m) {  // weights below tau are below min-p's (2^-18: the polynomial's slack)
          const unsigned long long wt = weight(tau, M, s);
          covered = wt + (wt >> 18) + 1 < kept.least;
        } else {
          covered = L >= max(1ull, draw_threshold(p_clamped, Z));
        }
      }
      if (covered) {
        if (c.rank == 0) {
          // ---- 3. the cuts and the draw on the list ----
          unsigned long long key[kPerThread], w[kPerThread], one[kPerThread], id[kPerThread];
#pragma unroll
          for (int i = 0; i < kPerThread; ++i) {
            const int e = i * kThreadsS + tid;
            const bool in = e < listed;
            const uint2 q = in ? list[e] : make_uint2(0, 0);
            const float x = __uint_as_float(q.x);
            key[i] = cut_key(x, q.y);
            id[i] = q.y;
            one[i] = in;
            w[i] = in ? weight(x, M, s) : 0ull;
            if (w[i] < kept.least) w[i] = 0;
          }
          const unsigned long long klo = cut_key(M, 0), khi = cut_key(from, 0x3fffff);
          if (has_k && set.k < listed) {
            kept.cut = list_crossing<true>(c, key, one, klo, khi, set.k - 1);
#pragma unroll
            for (int i = 0; i < kPerThread; ++i)
              if (key[i] > kept.cut) w[i] = 0;
          }
          if (has_p) {
            unsigned long long total = 0;
#pragma unroll
            for (int i = 0; i < kPerThread; ++i) total += w[i];
            total = whole ? Z : block_sum(total, sh.part);
            kept.cut = list_crossing<false>(c, key, w, klo, khi, max(1ull, draw_threshold(p_clamped, total)) - 1);
#pragma unroll
            for (int i = 0; i < kPerThread; ++i)
              if (key[i] > kept.cut) w[i] = 0;
          }
          unsigned long long t = 0, n_kept = 0, top = 0;
#pragma unroll
          for (int i = 0; i < kPerThread; ++i) {
            t += w[i];
            n_kept += w[i] > 0;
            if (w[i] && key[i] > top) top = key[i];
          }
          block_sum2(t, n_kept, sh, &S, &count);
          if (a.filtered) {  // the largest key kept: a bound for rows cut by min-p alone
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            __syncthreads();
            if (lane == 0) sh.part[warp] = top;
            __syncthreads();
#pragma unroll
            for (int x = 0; x < kWarpsS; ++x) top = max(top, sh.part[x]);
            kept.cut = top;
          }
          token = static_cast<int>(list_crossing<false>(c, id, w, 0, a.V - 1, draw_threshold(u, S)));
#pragma unroll
          for (int i = 0; i < kPerThread; ++i)
            if (w[i] && id[i] == static_cast<unsigned long long>(token)) sh.part2[0] = w[i];
          __syncthreads();
          if (tid == 0) {
            a.tokens[row] = token;
            if (a.p) a.p[row] = __fdiv_rn(__ull2float_rn(sh.part2[0]), __ull2float_rn(S));
            if (a.n_kept) a.n_kept[row] = static_cast<int>(count);
          }
          if (a.filtered && tid < c.C) *c.at(&sh.cut, tid) = kept.cut;
        }
        if (a.filtered) {
          c.sync();
          kept.cut = sh.cut;
        }
      } else {
        // ---- the cuts over the slices ----
        auto cut_at = [&](unsigned long long key) {
          kept.cut = key;
          edge = logit_of(key);
        };
        if (has_k)
          cut_at(slice_crossing<E, kStaged, true>(c, sl, M, s, set.k - 1, weigh));
        if (has_p) {
          unsigned long long total = Z;
          if (!(whole && lists)) {
            c.sync();  // the list is not read any more
            group_sums<E, kStaged>(c, sl, groups, [&](int v, unsigned int* k) {
              const uint4 x = sl.at(v);
              unsigned long long t = 0;
#pragma unroll
              for (int i = 0; i < VEC; ++i) t += weigh(sl.first + v * VEC + i, element<E>(x, i));
              return t;
            }, &total, &count);
          }
          cut_at(slice_crossing<E, kStaged, false>(c, sl, M, s, max(1ull, draw_threshold(p_clamped, total)) - 1, weigh));
        }
      }
    }
    if (!covered) {
      // ---- the draw over the slices ----
      c.sync();  // the list is not read any more
      const bool all = !(has_k || has_m || has_p);
      group_sums<E, kStaged>(c, sl, groups, [&](int v, unsigned int* k) {
        const uint4 w = sl.at(v);
        if (all) {
          Sum z;
          float2 x[VEC / 2];
          unpack_pairs<E>(w, x);
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) {
            const float2 y = add_pair(z, x[i], M, s, mz);
            *k += (y.x > 0.5f) + (y.y > 0.5f);
          }
          return value_of(z, VEC);
        }
        unsigned long long t = 0;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const unsigned long long e = weigh(sl.first + v * VEC + i, element<E>(w, i));
          t += e;
          *k += e > 0;
        }
        return t;
      }, &S, &count);
      token = group_draw<E, kStaged>(c, sl, groups, draw_threshold(u, S), weigh);
      if (token >= 0) {  // on the rank that holds it
        const float x_token = kStaged ? staged_elem<E>(slice, token - sl.first) : load_one<E>(sl.global, token - sl.first);
        if (tid == 0) {
          a.tokens[row] = token;
          if (a.p) a.p[row] = __fdiv_rn(__ull2float_rn(weight(x_token, M, s)), __ull2float_rn(S));
          if (a.n_kept) a.n_kept[row] = static_cast<int>(count);
        }
      }
    }
  } else if (c.rank == 0 && tid == 0) {
    a.tokens[row] = 0;
    if (a.p) a.p[row] = 0.f;
    if (a.n_kept) a.n_kept[row] = 0;
  }

  // ---- the filtered row ----
  if (a.filtered) {
    edge = good ? logit_of(kept.cut) : INFINITY;
    if (!good) kept.cut = 0;
    for (int v = tid; v < sl.nv; v += kThreadsS)
      write_kept<E>(a, row, sl.first, v, sl.at(v), aligned_out && sl.first + (v + 1) * VEC <= a.V, kept, edge, M, s);
  }
  if (tid == 0) {
    int bad = timeout ? kWaitTimeout : 0;
    if (c.rank == 0) {
      bad |= set.bad | (good ? 0 : kDataNonfiniteLogit);
      if (!(u >= 0.f && u < 1.f)) bad |= kDataUniformRange;
    }
    if (bad && a.status) atomicOr(a.status, bad);
  }
}

// Blocks per row: the fewest whose slices fit, or 8 that read global memory.
struct Shape {
  int nvec, C, nvs;
  bool staged;
};
Shape shape_of(int V, bool bf16) {
  Shape s;
  s.nvec = (V + (bf16 ? 8 : 4) - 1) / (bf16 ? 8 : 4);
  for (s.C = 1; s.C <= kMaxCS; s.C *= 2) {
    s.nvs = (s.nvec + s.C - 1) / s.C;
    if (s.nvs * 16ll <= (s.C == kMaxCS ? kMaxSliceS : kSliceBytesS)) {
      s.staged = true;
      return s;
    }
  }
  s.C = kMaxCS;
  s.nvs = 0;
  s.staged = false;
  return s;
}

constexpr size_t kTailBytes = kList * 8 + kDepth * kThreadsS * 2;
static_assert(kDepth * kThreadsS * 2 >= static_cast<int>(sizeof(Bins)), "the bins fit the threads' lists");

template <typename E, bool kStaged>
cudaError_t launch(const SampleArgs& a, const Shape& s, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned int>(a.R) * s.C);
  cfg.blockDim = dim3(kThreadsS);
  cfg.dynamicSmemBytes = static_cast<size_t>(s.nvs) * 16 + kTailBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = s.C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool in = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && a.row_stride * E::kBytes % 16 == 0 &&
                  a.V % Staged<E>::kVec == 0;
  const bool out = reinterpret_cast<uintptr_t>(a.filtered) % 16 == 0 && a.V % Staged<E>::kVec == 0;
  return cudaLaunchKernelEx(&cfg, filtered_sample_kernel<E, kStaged>, a, s.nvec, s.nvs, in, out, -0.f);
}

}  // namespace

size_t filtered_sample_workspace(int R, int V, bool bf16) {
  (void)R;
  (void)V;
  (void)bf16;
  return 0;
}

cudaError_t filtered_sample_prepare() {
  const int bytes = static_cast<int>(kMaxSliceS + kTailBytes);
  cudaError_t e = cudaFuncSetAttribute(filtered_sample_kernel<BF16, true>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(filtered_sample_kernel<F32, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  return e;
}

cudaError_t launch_filtered_sample(const SampleArgs& a, void* ws, int sm_count, cudaStream_t stream) {
  (void)ws;
  (void)sm_count;
  const Shape s = shape_of(a.V, a.bf16);
  if (a.bf16) return s.staged ? launch<BF16, true>(a, s, stream) : launch<BF16, false>(a, s, stream);
  return s.staged ? launch<F32, true>(a, s, stream) : launch<F32, false>(a, s, stream);
}

}  // namespace specv
