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
// Four kernels:
//   list    one cluster of C blocks per row, each block's slice in shared
//           memory (TMA bulk copies), so the row crosses HBM once.  As the
//           copies land every thread keeps its largest logit; the cluster
//           exchanges the row's maximum and a threshold, a quantile of the
//           threads' maxima above which some hundred logits lie (or min-p's
//           own threshold where that is higher).  One sweep over the slice
//           lists the logits from there up and, when top-p asks for a share
//           of the whole row's mass, sums approximate weights of the others
//           with a bound on the error.  What a cut keeps nearly always lies in
//           the list -- the k largest, what min-p leaves, the share that top-p
//           asks for -- and whether it does is known from counts and sums.
//           Rows without cuts are drawn here, from exact sums by 32-vector
//           group.
//   finish  one small block per listed row makes the cuts and the draw on it.
//           The cut that the approximate sum gives is checked against the
//           sum's bounds.
//   whole   a cluster does all of a row's work at once.  It takes the rows that
//           the first two queue -- those whose kept set does not lie in the
//           list (flat distributions), by bins over the slices, and the rare
//           ones between the bounds (its own sums are exact) -- and every row of a
//           call whose clusters all fit the GPU at once, where latency counts
//           and there is no next row to overlap.
//   write   filtered rows that take the logits' place, streaming.  (Others are
//           filled with -inf by the list kernel, on its way, and finish adds
//           what is kept.)
//
// Measured, bf16: 4096 rows of 32000, top-p 0.9, 171 us, of which list 95 (the
// logits at the copy rate: 39; 17 instructions a logit at two thirds of the
// issue slots), finish 46 (lists of 845 entries in three passes), whole 29 for
// the few rows between the bounds (one row's latency); 384 rows of 128256 with
// eight settings and filtered rows 81 us (30; the list kernel's 58 with 40 % of
// the issue slots and 30 % of DRAM in use: barriers and latency); 4 rows of
// 1000 in the whole kernel alone 12.  Rows whose kept set is wider than the
// list go one by one through the whole kernel: 4096 rows of 32000 that keep
// 1445 each take 1.7 ms (39), and a flat row that keeps a tenth of its 32000
// logits takes a cluster 100 us.  Rows off 16 bytes are loaded by element:
// 4096 of 32001 320 us.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <cfloat>
#include <climits>

#include "device_common.cuh"
#include "launch_decode.h"
#include "sample_common.cuh"

namespace cg = cooperative_groups;

namespace specv {
namespace {

constexpr int kThreadsS = 256;          // row kernel
constexpr int kWarpsS = kThreadsS / 32;
constexpr int kThreadsB = 128;          // finish kernel
constexpr int kMaxCS = 8;               // blocks of a cluster
constexpr int kList = 1536;             // listed logits of a row
constexpr int kLongList = 4095;         // of a queued row (bins hold 4095 of the largest weight)
constexpr int kPlaces = 4096;           // of a block, as 16-bit places in its slice
constexpr int kGroupSums = 1024;        // group sums of a block (they share the places' memory)
constexpr int kGroups = kGroupSums / kWarpsS;  // rounds with group sums of their own 
constexpr long long kSliceBytesS = 65024;     // a slice, while more blocks can share the row
constexpr long long kMaxSliceS = 128 * 1024;  // a slice of the largest cluster (with a long list beside it)
constexpr int kChunkS = 1024;           // vectors per bulk copy
constexpr int kMaxChunksS = 8;         // (65536 bf16 of a slice: 16-bit places)
static_assert(kMaxSliceS / 16 <= kChunkS * kMaxChunksS, "bulk copies of a slice");
constexpr int kVectorsS = (kMaxSliceS / 16 + kThreadsS - 1) / kThreadsS;  // vectors of a slice a thread sweeps at most
// Blocks of the row kernel that run at once (two an SM, 152 SMs): rows in
// clusters of no more than these are finished in it.  A constant, so that a
// workspace's size does not depend on the device; nothing waits for as many to
// run at once.
constexpr int kFusedBlocks = 304;
constexpr int kRowsAtOnce = 4096;       // rows listed in the workspace at a time

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

// Which tokens are kept: key (falling logit, index) at most `cut`, weight at
// least `least` (weight 0 is never kept).
struct Kept {
  unsigned long long cut, least;
};
// A bf16 has 16 bits of its own, which leaves the key's bins to them and the index.
template <typename E>
__device__ __forceinline__ unsigned int value_key(float x) {
  return E::kBytes == 2 ? falling(x) >> 16 : falling(x);
}
template <typename E>
__device__ __forceinline__ unsigned long long cut_key(float x, unsigned int j) {
  return (static_cast<unsigned long long>(value_key<E>(x)) << 22) | j;
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

// Which elements of a vector are at least a threshold, the vector with -inf
// in their place, and the place of the element behind a bit.  bf16 compares
// pairs against the smallest bf16 that is no less than the threshold (bits
// 0-3 even elements, 4-7 odd ones).
template <typename E>
struct AtLeast;
template <>
struct AtLeast<F32> {
  float from;
  __device__ __forceinline__ explicit AtLeast(float f) : from(f) {}
  __device__ __forceinline__ uint32_t bits(uint4& w) const {
    uint32_t u[4] = {w.x, w.y, w.z, w.w}, t = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (__uint_as_float(u[k]) >= from) {
        t |= 1u << k;
        u[k] = 0xff800000u;
      }
    w = make_uint4(u[0], u[1], u[2], u[3]);
    return t;
  }
  // the other way round: -inf in place of the others; and the test alone
  __device__ __forceinline__ uint32_t keep(uint4& w) const {
    const uint32_t t = which(w);
    w = make_uint4(t & 1 ? w.x : 0xff800000u, t & 2 ? w.y : 0xff800000u, t & 4 ? w.z : 0xff800000u,
                   t & 8 ? w.w : 0xff800000u);
    return t;
  }
  __device__ __forceinline__ uint32_t which(const uint4& w) const {
    return (__uint_as_float(w.x) >= from ? 1u : 0u) | (__uint_as_float(w.y) >= from ? 2u : 0u) |
           (__uint_as_float(w.z) >= from ? 4u : 0u) | (__uint_as_float(w.w) >= from ? 8u : 0u);
  }
  static __device__ __forceinline__ int place(int bit) { return bit; }
};
template <>
struct AtLeast<BF16> {
  __nv_bfloat162 from;
  __device__ __forceinline__ explicit AtLeast(float f) { from = __bfloat162bfloat162(__float2bfloat16_ru(f)); }
  __device__ __forceinline__ uint32_t bits(uint4& w) const {
    uint32_t u[4] = {w.x, w.y, w.z, w.w}, t = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t m = mask(u[k]);
      t |= m & (0x00010001u << k);
      u[k] = (u[k] & ~m) | (m & 0xff80ff80u);
    }
    w = make_uint4(u[0], u[1], u[2], u[3]);
    return (t | (t >> 12)) & 0xffu;
  }
  __device__ __forceinline__ uint32_t keep(uint4& w) const {
    uint32_t u[4] = {w.x, w.y, w.z, w.w}, t = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t m = mask(u[k]);
      t |= m & (0x00010001u << k);
      u[k] = (u[k] & m) | (~m & 0xff80ff80u);
    }
    w = make_uint4(u[0], u[1], u[2], u[3]);
    return t;
  }
  __device__ __forceinline__ uint32_t which(const uint4& w) const {
    return (mask(w.x) & 0x00010001u) | (mask(w.y) & 0x00020002u) | (mask(w.z) & 0x00040004u) |
           (mask(w.w) & 0x00080008u);
  }
  __device__ __forceinline__ uint32_t mask(uint32_t u) const {
    __nv_bfloat162 x;
    memcpy(&x, &u, 4);
    return __hge2_mask(x, from);
  }
  static __device__ __forceinline__ int place(int bit) { return ((bit & 3) << 1) | (bit >> 2); }
};

// The approximate mass of a vector, sum of 2^t by ex2.approx.
template <typename E>
__device__ __forceinline__ float vector_mass(const uint4& w, float M, float s, float mz) {
  constexpr int NP = Staged<E>::kVec / 2;
  float2 x[NP];
  unpack_pairs<E>(w, x);
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const float2 t = fmul2(fadd2(x[k], both(-M)), both(s), mz);
    x[k] = make_float2(ex2(t.x), ex2(t.y));
  }
#pragma unroll
  for (int h = NP / 2; h > 0; h >>= 1)
#pragma unroll
    for (int k = 0; k < h; ++k) x[k] = fadd2(x[k], x[k + h]);
  return x[0].x + x[0].y;
}

// The logit of a cut key; the lowest finite one for "no cut".
template <typename E>
__device__ __forceinline__ float logit_of(unsigned long long cut) {
  if (cut == ~0ull) return -FLT_MAX;
  if constexpr (E::kBytes == 2) {
    const unsigned int o = ~static_cast<unsigned int>(cut >> 22) & 0xffffu;
    return __uint_as_float(((o >> 15) ? o & 0x7fffu : ~o & 0xffffu) << 16);
  } else {
    const unsigned int o = ~static_cast<unsigned int>(cut >> 22);
    return __uint_as_float((o >> 31) ? o & 0x7fffffffu : ~o);
  }
}

// What every rank of a cluster publishes to all.
struct Exchange {
  float max[kMaxCS], tau[kMaxCS];  // tau: sum of the warps' order statistics, taus of them
  int taus[kMaxCS], listed[kMaxCS];  // taus -1: a copy never landed
  unsigned long long sum[kMaxCS], listed_sum[kMaxCS];
  unsigned long long mass[kMaxCS], count[kMaxCS];
};

// Scratch of block-wide steps.
struct Shared {
  unsigned long long part[16], part2[16];  // a warp each
  unsigned long long few_key[32], few_w[32];
  unsigned long long rem, lo, cut, w_token;
  unsigned int n_few, bin_count, list_n, taken;
  int sel[2];
  float wmax[16], wtau[16];
  Settings set;
  float u, s;
  unsigned long long least;
  int lane_of_tau;
  int stuck;  // copies never landed: the barriers' phases are lost, so no later row is copied
};

// 256 bins of weights, kept as 32-bit parts so that shared memory adds them
// without a loop, and of counts.
struct ListBins {
  unsigned int count[256], part[2][256];
};
struct Bins {  // begins as ListBins does
  unsigned int count[256], part[4][256];
  unsigned long long sum[256];  // of the cluster
  unsigned int all[256];
};
template <int kParts>  // parts of 20 bits (a list: less than 2^12 of the largest weight) or of 11 (a slice)
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
  Exchange* x;
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
  // kParts of the bins' parts and the counts to zero.
  template <int NT, int kParts>
  __device__ __forceinline__ void clear() const {
    for (int i = threadIdx.x; i < 256; i += NT) {
#pragma unroll
      for (int k = 0; k < kParts; ++k) bins->part[k][i] = 0;
      bins->count[i] = 0;
    }
    if (threadIdx.x == 0) sh->n_few = 0;
  }
};

// Two block-wide sums at once.
template <int NT>
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
  for (int w = 0; w < NT / 32; ++w) {
    *sa += sh.part[w];
    *sb += sh.part2[w];
  }
}

// One warp: the first of 256 bins (by the running sum of value(bin)) to pass
// rem.  Leaves the bin, what is left of rem inside it and its count in `sh`.
template <typename F>
__device__ __forceinline__ void crossing_bin(const Ctx& c, unsigned long long rem, F value,
                                             const unsigned int* counts) {
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
    c.sh->bin_count = counts[lane * 8 + b];
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

// A listed logit: its bits, its index, its weight's low 20 bits and the rest.
__device__ __forceinline__ uint4 make_entry(float x, unsigned int j, unsigned long long w) {
  return make_uint4(__float_as_uint(x), j, static_cast<unsigned int>(w) & 0xfffffu, static_cast<unsigned int>(w >> 20));
}
__device__ __forceinline__ unsigned long long weight_of(const uint4& e) {
  return (static_cast<unsigned long long>(e.w) << 20) + e.z;
}
template <typename E>
__device__ __forceinline__ unsigned long long key_of(const uint4& e) { return cut_key<E>(__uint_as_float(e.x), e.y); }

// The crossing key over n listed elements by a block of NT threads.  keys(entry) lie in
// [lo, hi]; measure(entry) is an element's weight (kCount: 0 or 1).
template <int NT, bool kCount, typename K, typename F>
__device__ __forceinline__ unsigned long long list_crossing(const Ctx& c, const uint4* list, int n, unsigned long long lo,
                                                            unsigned long long hi, unsigned long long rem, K keys,
                                                            F measure) {
  int shift = bin_shift(hi - lo);
  for (;;) {
    __syncthreads();
    c.clear<NT, kCount ? 0 : 2>();
    __syncthreads();
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += NT) {
      const uint4 e = list[i];
      const unsigned long long at = (keys(e) - lo) >> shift, w = measure(e);
      if (w && at < 256) {  // (a key below lo wraps to a large bin)
        if (kCount) atomicAdd(&c.bins->count[at], 1u);
        else bin_add<2>(c.bins, static_cast<unsigned int>(at), w);
      }
    }
    __syncthreads();
    if (threadIdx.x < 32)
      crossing_bin(c, rem, [&](int b) -> unsigned long long {
        return kCount ? c.bins->count[b] : bin_value<2>(c.bins, b);
      }, c.bins->count);
    __syncthreads();
    rem = c.sh->rem;
    lo += static_cast<unsigned long long>(c.sh->sel[0]) << shift;
    if (shift == 0) return lo;
    if (c.sh->bin_count <= 32) break;
    shift = shift > 8 ? shift - 8 : 0;
  }
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += NT) {
    const uint4 e = list[i];
    const unsigned long long key = keys(e), w = measure(e);
    if (w && (key - lo) >> shift == 0) {
      const unsigned int at = atomicAdd(&c.sh->n_few, 1u);
      if (at < 32) {
        c.sh->few_key[at] = key;
        c.sh->few_w[at] = w;
      }
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
    c.clear<kThreadsS, kCount ? 0 : 4>();
    __syncthreads();
    sweep(from, to, [&](unsigned int j, float x) {
      unsigned int at = bin_of(x);
      if (shift >= 0) {
        const unsigned long long key = cut_key<E>(x, j), d = (key - lo) >> shift;
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
    if (threadIdx.x < 32) crossing_bin(c, rem, [&](int b) { return c.bins->sum[b]; }, c.bins->all);
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
      lo = cut_key<E>(to, 0);
      shift = bin_shift(cut_key<E>(from, 0x3fffff) - lo);
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
    const unsigned long long key = cut_key<E>(x, j);
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
  block_sum2<kThreadsS>(mine, n, *c.sh, &t, &k);
  if (threadIdx.x < c.C) {
    *c.at(&c.x->mass[c.rank], threadIdx.x) = t;
    *c.at(&c.x->count[c.rank], threadIdx.x) = k;
  }
  c.sync();
  *S = *count = 0;
  for (int r = 0; r < c.C; ++r) {
    *S += c.x->mass[r];
    *count += c.x->count[r];
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
    if (off + c.x->mass[r] > theta) {
      owner = r;
      break;
    }
    off += c.x->mass[r];
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
    int token = sl.first;
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
__device__ __forceinline__ int tau_lane(const Settings& set, int V, int C, int most) {
  const float share = 0.55f * most;  // room for rows that list more than meant
  const float m = set.k < V ? fminf(1.25f * set.k + 64.f, share) : share;
  const float below = ex2(-1.44269504f * m / (kThreadsS * C));
  return min(31, max(0, static_cast<int>(32.f * below)));
}

// Below the first logit every weight is 0, from the second up 1 or more: a
// weight is 1 from 2^-41 of the largest up, and t, the polynomial and these
// logits are off by less than 1e-4 and |M| 2^-22.
__device__ __forceinline__ float zero_logit(float M, float s) { return M - __fdiv_rn(41.001f, s) - fabsf(M) * 2.4e-7f; }
__device__ __forceinline__ float sure_logit(float M, float s) {
  return fmaxf(M - __fdiv_rn(40.999f, s) + fabsf(M) * 2.4e-7f, -FLT_MAX);
}

// A vector of the filtered row.  Nearly every element is below `edge` and not
// kept, or from `sure` (NaN: none) up and kept; the others are tested exactly.
template <typename E>
__device__ __forceinline__ void write_kept(const SampleArgs& a, int row, int first, int v, const uint4& w,
                                           bool vectors, const Kept& kept, float edge, float sure, float M, float s) {
  constexpr int VEC = Staged<E>::kVec;
  using raw = typename E::raw;
  uint4 o = w;
  AtLeast<E> above(edge), certain(sure);
  const uint32_t some = above.keep(o);
  if (some != certain.which(w)) {
    raw x[VEC];
    memcpy(x, &w, 16);
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const float f = element<E>(w, k);
      bool in = f >= edge;
      if (in && !(f >= sure)) in = cut_key<E>(f, first + v * VEC + k) <= kept.cut && weight(f, M, s) >= kept.least;
      if (!in) x[k] = masked_value<E>();
    }
    memcpy(&o, x, 16);
  }
  raw* dst = static_cast<raw*>(a.filtered) + static_cast<size_t>(row) * a.V + first + v * VEC;
  if (vectors) {
    *reinterpret_cast<uint4*>(dst) = o;
  } else {
    raw x[VEC];
    memcpy(x, &o, 16);
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      if (first + v * VEC + k < a.V) dst[k] = x[k];
  }
}

// -inf over `n` elements of the filtered row from `first` on: 16-byte stores,
// and single elements at ends that are not on 16 bytes.
template <typename E>
__device__ __forceinline__ void fill_masked(const SampleArgs& a, int row, int first, int n) {
  using raw = typename E::raw;
  const int tid = threadIdx.x;
  n = min(n, a.V - first);
  raw* to = static_cast<raw*>(a.filtered) + static_cast<size_t>(row) * a.V + first;
  const int lead = min(n, static_cast<int>(-reinterpret_cast<uintptr_t>(to) & 15u) / E::kBytes);
  const int vectors = (n - lead) * E::kBytes / 16, done = lead + vectors * (16 / E::kBytes);
  if (tid < lead) to[tid] = masked_value<E>();
  if (tid < n - done) to[done + tid] = masked_value<E>();
  const uint32_t inf = E::kBytes == 2 ? 0xff80ff80u : 0xff800000u;
  uint4* at = reinterpret_cast<uint4*>(to + lead);
#pragma unroll 4
  for (int v = tid; v < vectors; v += kThreadsS) __stcs(at + v, make_uint4(inf, inf, inf, inf));
}

// A row on its way between the kernels.
struct __align__(16) RowHead {
  float M, from;                 // largest logit, smallest listed one
  unsigned long long Z, slack;   // mass of the row (2^-40) and how far the exact sum may be from it, for top-p
  unsigned long long cut;        // kept keys go up to here (for the write kernel)
  int listed;                    // -1: nothing to finish
  int good;
  int written;                   // the filtered row is (being) written by the whole-row kernel
};

// Rows for the whole-row kernel.  Zero at rest: its last block puts it back.
struct __align__(16) Queue {
  unsigned int n, readers;
};

// How far the exact sum of the unlisted weights can be from the approximate
// one, U.  The approximate terms are 2^t of the same t by ex2.approx (2^-22.5
// off) instead of the polynomial (2^-22.3), summed in fp32 by at most ten
// additions (2^-20.7): together below 2^-20; and each of at most V
// whole-number weights is rounded by 1/2.
__device__ __forceinline__ unsigned long long sum_slack(unsigned long long U, int V) { return (U >> 20) + V; }

__device__ __forceinline__ unsigned long long share_of(float top_p, unsigned long long total) {
  return max(1ull, draw_threshold(fminf(fmaxf(top_p, 0.f), 0.99999994f), total));
}

// The cuts and the draw of a covered row on its list by a block of NT threads.  Writes
// the row's outputs; returns the largest kept key (~0 when the row needs
// its exact sum).  Three passes over the list: weights by bins of the logit's bits (top-p); sums of what lies above
// the crossing bin, by bins of the index; the crossing bin of the draw.  A
// bin of more than 32 candidates (ties) goes through list_crossing.
template <typename E, int NT>
__device__ unsigned long long finish_row(const Ctx& c, const SampleArgs& a, const Settings& set,
                                         unsigned long long least, float u, int row, const uint4* list,
                                         const RowHead& head, float s) {
  const bool has_k = set.k < a.V, has_m = set.min_p > 0.f, has_p = set.top_p < 1.f, whole = !has_k && !has_m;
  const int n = head.listed, tid = threadIdx.x;
  const unsigned int f0 = value_key<E>(head.M);
  const int fshift = bin_shift(value_key<E>(head.from) - f0), jshift = bin_shift(a.V - 1);
  const unsigned long long klo = cut_key<E>(head.M, 0), khi = cut_key<E>(head.from, 0x3fffff);
  ListBins* by_index = reinterpret_cast<ListBins*>(c.bins) + 1;
  unsigned long long cut = ~0ull;
  auto kept = [&](const uint4& e) -> unsigned long long {
    const unsigned long long w = weight_of(e);
    return w >= least && key_of<E>(e) <= cut ? w : 0ull;
  };
  if (has_k && set.k < n)
    cut = list_crossing<NT, true>(c, list, n, klo, khi, set.k - 1, key_of<E>, [](const uint4&) { return 1ull; });
  const unsigned long long slack = whole ? head.slack : 0;
  unsigned long long total = head.Z;
  if (has_p && !whole) {
    unsigned long long t = 0, k;
    for (int i = tid; i < n; i += NT) t += kept(list[i]);
    block_sum2<NT>(t, 0, *c.sh, &total, &k);
  }
  unsigned long long S, count;
  // ---- top-p: the crossing bin ----
  int bin = 256;  // kept for sure: bins below
  unsigned long long rem = 0;
  if (has_p) {
    rem = share_of(set.top_p, total - slack) - 1;
    __syncthreads();
    c.clear<NT, 2>();
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < n; i += NT) {
      const uint4 e = list[i];
      if (kept(e)) {
        const unsigned int at = min(255u, (value_key<E>(__uint_as_float(e.x)) - f0) >> fshift);
        atomicAdd(&c.bins->part[0][at], e.z);
        atomicAdd(&c.bins->part[1][at], e.w);
        atomicAdd(&c.bins->count[at], 1u);
      }
    }
    __syncthreads();
    if (tid < 32)
      crossing_bin(c, rem, [&](int b) { return bin_value<2>(c.bins, b); }, c.bins->count);
    __syncthreads();
    bin = c.sh->sel[0];
    rem = c.sh->rem;
    if (c.sh->bin_count > 32) {
      const unsigned long long lo = static_cast<unsigned long long>(f0 + (static_cast<unsigned int>(bin) << fshift)) << 22;
      cut = list_crossing<NT, false>(c, list, n, lo, lo + (1ull << (fshift + 22)) - 1, rem, key_of<E>, kept);
      bin = 256;
    }
  }
  // ---- what is kept, by bins of the index ----
  __syncthreads();
  for (int i = tid; i < 256; i += NT) by_index->count[i] = by_index->part[0][i] = by_index->part[1][i] = 0;
  if (tid == 0) c.sh->n_few = 0;
  __syncthreads();
  unsigned long long t = 0;
  unsigned int k = 0;
  auto add = [&](unsigned int j, unsigned int lo, unsigned int hi) {
    const unsigned int at = j >> jshift;
    atomicAdd(&by_index->part[0][at], lo);
    atomicAdd(&by_index->part[1][at], hi);
    atomicAdd(&by_index->count[at], 1u);
    t += (static_cast<unsigned long long>(hi) << 20) + lo;
    ++k;
  };
#pragma unroll 4
  for (int i = tid; i < n; i += NT) {
    const uint4 e = list[i];
    if (!kept(e)) continue;
    const int at = static_cast<int>(min(255u, (value_key<E>(__uint_as_float(e.x)) - f0) >> fshift));
    if (at < bin) {
      add(e.y, e.z, e.w);
    } else if (at == bin) {
      const unsigned int f = atomicAdd(&c.sh->n_few, 1u);
      if (f < 32) {
        c.sh->few_key[f] = key_of<E>(e);
        c.sh->few_w[f] = weight_of(e);
      }
    }
  }
  if (bin < 256) {
    __syncthreads();
    if (tid < 32) {
      const int few = min(32u, c.sh->n_few);
      const unsigned long long key = crossing_of_few(c.sh->few_key, c.sh->few_w, few, rem);
      if (tid < few && c.sh->few_key[tid] <= key)
        add(static_cast<unsigned int>(c.sh->few_key[tid]) & 0x3fffffu,
            static_cast<unsigned int>(c.sh->few_w[tid]) & 0xfffffu, static_cast<unsigned int>(c.sh->few_w[tid] >> 20));
      if (tid == 0) c.sh->lo = key;
    }
    __syncthreads();
    cut = c.sh->lo;
  }
  block_sum2<NT>(t, k, *c.sh, &S, &count);
  // the kept mass reaches the smallest share that the approximate sum
  // allows; if it does not reach the largest, the whole-row kernel takes the row
  if (has_p && slack != 0 && S < share_of(set.top_p, total + slack)) return ~0ull;
  // ---- the draw ----
  const unsigned long long theta = draw_threshold(u, S);
  __syncthreads();
  if (tid < 32) {
    crossing_bin(c, theta, [&](int b) {
      return (static_cast<unsigned long long>(by_index->part[1][b]) << 20) + by_index->part[0][b];
    }, by_index->count);
    if (tid == 0) c.sh->n_few = 0;
  }
  __syncthreads();
  unsigned long long token;
  if (c.sh->bin_count <= 32) {
    const unsigned int at = static_cast<unsigned int>(c.sh->sel[0]);
    const unsigned long long rem = c.sh->rem;
#pragma unroll 4
    for (int i = tid; i < n; i += NT) {
      const uint4 e = list[i];
      if (e.y >> jshift == at && kept(e)) {
        const unsigned int f = atomicAdd(&c.sh->n_few, 1u);
        if (f < 32) {
          c.sh->few_key[f] = e.y;
          c.sh->few_w[f] = weight_of(e);
        }
      }
    }
    __syncthreads();
    if (tid < 32) {
      const int few = min(32u, c.sh->n_few);
      token = crossing_of_few(c.sh->few_key, c.sh->few_w, few, rem);
      if (tid < few && c.sh->few_key[tid] == token) c.sh->w_token = c.sh->few_w[tid];
      if (tid == 0) c.sh->lo = token;
    }
    __syncthreads();
    token = c.sh->lo;
  } else {
    token = list_crossing<NT, false>(c, list, n, 0, a.V - 1, theta,
                                     [](const uint4& e) -> unsigned long long { return e.y; }, kept);
    for (int i = tid; i < n; i += NT)
      if (list[i].y == token) c.sh->w_token = weight_of(list[i]);
    __syncthreads();
  }
  unsigned long long top = a.filtered ? cut : 0;  // (only the filtered row needs it)
  if (top == ~0ull) {  // no cut by k or p: the largest key kept
    top = 0;
    for (int i = tid; i < n; i += NT)
      if (kept(list[i])) top = max(top, key_of<E>(list[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((tid & 31) == 0) c.sh->part[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < NT / 32; ++x) top = max(top, c.sh->part[x]);
  }
  if (tid == 0) {
    a.tokens[row] = static_cast<int>(token);
    if (a.p) a.p[row] = __fdiv_rn(__ull2float_rn(c.sh->w_token), __ull2float_rn(S));
    if (a.n_kept) a.n_kept[row] = static_cast<int>(count);
  }
  return top;
}

// A block that gave up on a row's copies waits for them once more, with the
// same limit: none may land after the block has left, or in the next row's
// slice.  True where some did not.
__device__ __noinline__ bool never_landed(unsigned long long* bars, int nch, uint32_t parity) {
  for (int k = 0; k < nch; ++k)
    if (!mbar_wait_sleep(&bars[k], parity)) return true;
  return false;
}

// The list kernel (kWhole false: cluster i takes row row0 + i) and the
// whole-row kernel (clusters take rows of the queue, or row i without one).
template <typename E, bool kStaged, bool kWhole>
__global__ void __launch_bounds__(kThreadsS, 3)
filter_row_kernel(const SampleArgs a, int row0, int nvec, int nvs, bool aligned_in, bool aligned_out, bool fill,
                  RowHead* heads, uint4* lists, int most, Queue* queue, int* queued, float mz) {
  constexpr int VEC = Staged<E>::kVec;
  constexpr int kPerWord = 32 / VEC, kWords = kStaged ? (kVectorsS + kPerWord - 1) / kPerWord : 1;
  using raw = typename E::raw;
  extern __shared__ __align__(128) uint4 dyn[];  // slice [nvs] | places, group sums or bins | list (kWhole)
  __shared__ Shared sh;
  __shared__ Exchange ex;
  __shared__ __align__(8) unsigned long long bars[kMaxChunksS];
  cg::cluster_group cluster = cg::this_cluster();
  Ctx c;
  c.sh = &sh;
  c.x = &ex;
  c.C = static_cast<int>(cluster.num_blocks());
  c.rank = static_cast<int>(cluster.block_rank());
  uint4* slice = dyn;
  uint16_t* places = reinterpret_cast<uint16_t*>(dyn + (kStaged ? nvs : 0));
  unsigned long long* groups = reinterpret_cast<unsigned long long*>(places);
  c.bins = reinterpret_cast<Bins*>(places);
  uint4* list = reinterpret_cast<uint4*>(places + kPlaces);
  const int lgC = __ffs(c.C) - 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int v0 = static_cast<int>((static_cast<long long>(nvec) * c.rank) >> lgC);
  Slice<E, kStaged> sl;
  sl.nv = static_cast<int>((static_cast<long long>(nvec) * (c.rank + 1)) >> lgC) - v0;
  sl.first = v0 * VEC;
  sl.V = a.V;
  sl.staged = slice;
  sl.width = kStaged ? 1 : max(1, (sl.nv + kThreadsS * kGroups - 1) / (kThreadsS * kGroups));
  const int nch = (sl.nv + kChunkS - 1) / kChunkS;
  const bool bulk = kStaged && aligned_in;
  if (tid == 0) sh.stuck = 0;
  if (bulk && tid == 0) {
    for (int k = 0; k < nch; ++k) mbar_init(&bars[k], 1);
    fence_barrier_init();
  }
  const int clusters = static_cast<int>(gridDim.x >> lgC);
  int at = static_cast<int>(blockIdx.x >> lgC), stop_at = at + 1;
  if (kWhole && queue) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    stop_at = static_cast<int>(queue->n);
    __syncthreads();
    if (tid == 0 && atomicAdd(&queue->readers, 1u) + 1u == gridDim.x) {  // everyone has read n
      queue->n = 0;
      queue->readers = 0;
    }
  }
  for (int turn = 0; at < stop_at; at += clusters, ++turn) {
    const int row = kWhole && queue ? queued[at] : row0 + at;
    const raw* logits = static_cast<const raw*>(a.logits) + row * a.row_stride;
    sl.global = logits + sl.first;

    // ---- the slice into shared memory -----------------------------------
    if (bulk) {
      if (tid == 0 && !(kWhole && sh.stuck)) {
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
    // how much of the row's list is taken
    unsigned int* taken = c.at(&sh.taken, 0);
    if (tid == 32) {  // the row's settings, while the copies are under way
      sh.list_n = 0;
      if (c.rank == 0) *taken = 0;
      sh.set = settings_of(a, row);
      sh.u = a.uniforms[row];
      sh.s = __fdiv_rn(1.44269502f, sh.set.T);
      sh.least = max(1ull, __float2ull_rn(__fmul_rn(fminf(fmaxf(sh.set.min_p, 0.f), 1.f), kScale)));
      sh.lane_of_tau = tau_lane(sh.set, a.V, c.C, most);
    }
    __syncthreads();
    const Settings set = sh.set;
    const float u = sh.u, s = sh.s;
    const bool has_k = set.k < a.V, has_m = set.min_p > 0.f, has_p = set.top_p < 1.f;
    const bool cuts = has_k || has_m || has_p, whole = !has_k && !has_m;  // whole: top-p of the whole row's mass
    if (c.C > 1) cluster_arrive_relaxed();  // matched before the first store to another block

    // ---- the row's maximum and the list's threshold ------------------------
    bool landed = !(kWhole && sh.stuck);
#ifdef SPEC_DEBUG
    // (a test's way to a wait that ran out: one NaN as the row's uniform, another for its turn in the queue)
    if (__float_as_uint(u) == (kWhole && queue ? 0x7fc0e000u : 0x7fc0d000u) + c.rank) landed = false;
#endif
    Peak<E> peak;
    if (bulk && landed) {
      for (int k = 0; k < nch; ++k) {
        if (!mbar_wait_sleep(&bars[k], turn & 1)) {
          landed = false;
          break;
        }
        const int stop = min((k + 1) * kChunkS, sl.nv);
#pragma unroll 4
        for (int v = k * kChunkS + tid; v < stop; v += kThreadsS) peak.take(slice[v]);
      }
    } else if (!bulk) {
      for (int v = tid; v < sl.nv; v += kThreadsS) peak.take(sl.at(v));
    }
    const float mine = peak.value();
    const bool odd = __any_sync(0xffffffffu, isnan(mine));
    const float sorted = warp_sort(mine, lane);
    const float order = __shfl_sync(0xffffffffu, sorted, sh.lane_of_tau);
    if (lane == 31) {
      sh.wmax[warp] = odd ? INFINITY : sorted;
      sh.wtau[warp] = order;
    }
    const int timeout = __syncthreads_or(!landed);
    if (timeout && bulk && tid == 0 && !sh.stuck) sh.stuck = never_landed(bars, nch, turn & 1);
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
      *c.at(&ex.max[c.rank], tid) = m;
      *c.at(&ex.tau[c.rank], tid) = t;
      *c.at(&ex.taus[c.rank], tid) = timeout ? -1 : n;
    }
    c.sync();
    float M = -INFINITY, tau = 0.f;
    int taus = 0;
    bool lost = false;  // the row has no result (every block of the cluster goes the same way)
    for (int r = 0; r < c.C; ++r) {
      lost |= ex.taus[r] < 0;
      M = fmaxf(M, ex.max[r]);
      tau += ex.tau[r];
      taus += ex.taus[r];
    }
    tau = taus ? fminf(tau / taus, M) : -INFINITY;
    M += 0.f;
    const bool good = !lost && M > -INFINITY && M < INFINITY;
    if (tid == 0) {
      int bad = timeout ? kWaitTimeout : 0;
      if (c.rank == 0 && !(kWhole && queue)) {  // (the list kernel has reported a queued row's data and settings)
        bad |= set.bad | (good || lost ? 0 : kDataNonfiniteLogit);
        if (!(u >= 0.f && u < 1.f)) bad |= kDataUniformRange;
      }
      if (bad && a.status) atomicOr(a.status, bad);
    }
    Kept kept;
    kept.cut = ~0ull;
    kept.least = sh.least;
    RowHead head;
    head.M = M;
    head.from = M;
    head.Z = head.slack = 0;
    head.listed = -1;
    head.good = good;
    head.written = 0;
    bool later = false;  // for the whole-row kernel

    if (good && cuts && kStaged) {
      // ---- list, and approximate sum of the rest ----
      // below `floor` every weight is 0, below `least_x` under min-p's share
      // (with room for the roundings of t and of the polynomial, and for
      // shares near 2^-40 of the weight itself)
      const float floor = zero_logit(M, s);
      const float share = has_m ? __log2f(fminf(set.min_p, 1.f)) - (set.min_p < 1e-6f ? 2.f : 1e-4f) : -42.f;
      const float least_x = fmaxf(floor, M + __fdiv_rn(share, s) - fabsf(M) * 2.4e-7f);
      const bool complete = !(tau > least_x);
      const float from = complete ? least_x : tau;
      const AtLeast<E> test(from);
      uint32_t hits[kWords];
      float z = 0.f, z_low = 0.f;
      unsigned long long exact = 0;  // (kWhole)
      int n = 0;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        hits[i] = 0;
        if (i * kPerWord * kThreadsS < sl.nv) {
          float zi = 0.f;
#pragma unroll
          for (int k = 0; k < kPerWord; ++k) {
            const int v = (i * kPerWord + k) * kThreadsS + tid;
            if (v < sl.nv) {
              uint4 w = slice[v];
              if (kWhole && whole) {
                Sum x;
                float2 pair[VEC / 2];
                unpack_pairs<E>(w, pair);
#pragma unroll
                for (int p = 0; p < VEC / 2; ++p) add_pair(x, pair[p], M, s, mz);
                exact += value_of(x, VEC);
              }
              hits[i] |= test.bits(w) << (k * VEC);
              if (!kWhole && whole) zi += vector_mass<E>(w, M, s, mz);
            }
          }
          // z + z_low is the sum without a further rounding
          const float t = __fadd_rn(z, zi), q = __fsub_rn(t, z);
          z_low += __fadd_rn(__fsub_rn(z, __fsub_rn(t, q)), __fsub_rn(zi, q));
          z = t;
          n += __popc(hits[i]);
        }
      }
      // each thread's place in the block's list, the block's in the row's
      int incl = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
      }
      int place = 0;
      if (lane == 31) place = static_cast<int>(atomicAdd(&sh.list_n, static_cast<unsigned int>(incl)));
      place = __shfl_sync(0xffffffffu, place, 31) + incl - n;
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        for (uint32_t h = hits[i]; h; h &= h - 1) {
          const int bit = __ffs(h) - 1;
          const int e = ((i * kPerWord + bit / VEC) * kThreadsS + tid) * VEC + AtLeast<E>::place(bit % VEC);
          if (place < kPlaces) places[place] = static_cast<uint16_t>(e);
          ++place;
        }
      __syncthreads();
      const int all = static_cast<int>(sh.list_n), fit = min(all, kPlaces);
      int before = 0;
      if (c.C > 1) {
        if (tid == 0) sh.sel[0] = static_cast<int>(atomicAdd(taken, static_cast<unsigned int>(all)));
        __syncthreads();
        before = sh.sel[0];
      }
      uint4* to = kWhole ? c.at(list, 0) : lists + static_cast<size_t>(at) * kList;
      unsigned long long zs = 0, ls = 0;
      for (int i = tid; i < fit && before + i < most; i += kThreadsS) {
        const int e = places[i];
        const float x = staged_elem<E>(slice, e);
        const unsigned long long w = weight(x, M, s);
        ls += w;
        to[before + i] = make_entry(x, static_cast<unsigned int>(sl.first + e), w);
      }
      if (whole)
        block_sum2<kThreadsS>(
            kWhole ? exact : __float2ull_rn(z * kScale) + static_cast<long long>(z_low * kScale), ls, sh, &zs, &ls);
      if (tid < c.C) {
        *c.at(&ex.sum[c.rank], tid) = zs;
        *c.at(&ex.listed_sum[c.rank], tid) = ls;
        *c.at(&ex.listed[c.rank], tid) = all;
      }
      c.sync();
      int total = 0;
      bool crowded = false;
      unsigned long long L = 0, U = 0;
      for (int r = 0; r < c.C; ++r) {
        crowded |= ex.listed[r] > kPlaces;
        total += ex.listed[r];
        U += ex.sum[r];
        L += ex.listed_sum[r];
      }
      // does the list hold all that can be kept?  (more than `most`, or a
      // block's kPlaces, did not fit, and the sums then mean nothing)
      head.from = from;
      head.slack = kWhole ? 0 : sum_slack(U, a.V);
      head.Z = kWhole ? U : L + U;  // (the exact sum has the listed ones in it)
      if (total <= most && !crowded &&
          (complete || (has_k ? total >= set.k : !has_m && L >= share_of(set.top_p, head.Z + head.slack))))
        head.listed = total;
      later = !kWhole && head.listed < 0;
    }
    if (kWhole && head.listed >= 0) {
      if (c.rank == 0) {
        kept.cut = finish_row<E, kThreadsS>(c, a, set, kept.least, u, row, list, head, s);
        if (a.filtered && tid < c.C) *c.at(&sh.cut, tid) = kept.cut;
      }
      if (a.filtered) {
        c.sync();
        kept.cut = sh.cut;
      }
    }
    if (good && head.listed < 0 && !later) {
      // ---- the cuts and the draw over the slices ----
      float edge = -FLT_MAX;  // the cut's logit
      auto weigh = [&](unsigned int j, float x) -> unsigned long long {
        if (!(x >= edge) || (kWhole && cut_key<E>(x, j) > kept.cut)) return 0ull;
        const unsigned long long w = weight(x, M, s);
        return w >= kept.least ? w : 0ull;
      };
      // one vector's kept weights
      auto vector_sum = [&](int v, unsigned int* k) -> unsigned long long {
        const uint4 w = sl.at(v);
        if (!kWhole || (kept.cut == ~0ull && !has_m)) {  // all of them
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
      };
      unsigned long long S = 0, count = 0;
      if (kWhole) {
        auto cut_at = [&](unsigned long long key) {
          kept.cut = key;
          edge = logit_of<E>(key);
        };
        if (has_k) cut_at(slice_crossing<E, kStaged, true>(c, sl, M, s, set.k - 1, weigh));
        if (has_p) {
          c.sync();
          group_sums<E, kStaged>(c, sl, groups, vector_sum, &S, &count);
          cut_at(slice_crossing<E, kStaged, false>(c, sl, M, s, share_of(set.top_p, S) - 1, weigh));
        }
      }
      c.sync();
      group_sums<E, kStaged>(c, sl, groups, vector_sum, &S, &count);
      const int token = group_draw<E, kStaged>(c, sl, groups, draw_threshold(u, S), weigh);
      if (token >= 0 && tid == 0) {  // on the rank that holds it
        const float x = kStaged ? staged_elem<E>(slice, token - sl.first) : load_one<E>(sl.global, token - sl.first);
        a.tokens[row] = token;
        if (a.p) a.p[row] = __fdiv_rn(__ull2float_rn(weight(x, M, s)), __ull2float_rn(S));
        if (a.n_kept) a.n_kept[row] = static_cast<int>(count);
      }
    } else if (!good && c.rank == 0 && tid == 0) {
      a.tokens[row] = 0;
      if (a.p) a.p[row] = 0.f;
      if (a.n_kept) a.n_kept[row] = 0;
    }

    if (!good) kept.cut = 0;
    if (kWhole || (fill && !cuts)) {
      if (a.filtered) {
        const float bound = good ? fmaxf(logit_of<E>(kept.cut), zero_logit(M, s)) : INFINITY;
        const float sure = cuts || !good ? NAN : sure_logit(M, s);
        for (int v = tid; v < sl.nv; v += kThreadsS)
          write_kept<E>(a, row, sl.first, v, sl.at(v), aligned_out && sl.first + (v + 1) * VEC <= a.V, kept, bound,
                        sure, M, s);
      }
      if (kWhole) c.sync();  // this row's memory is free
    }
    // (here, as a cluster's barrier waits for the stores before it)
    if (!kWhole && fill && cuts) fill_masked<E>(a, row, sl.first, sl.nv * VEC);
    if (!kWhole && c.rank == 0 && tid == 0) {
      if (later) queued[atomicAdd(&queue->n, 1u)] = row;
      head.cut = kept.cut;
      head.written = later;
      heads[at] = head;
    }
  }
}

// One block per listed row, the list in shared memory.
template <typename E>
__global__ void __launch_bounds__(kThreadsB, 8) filter_finish_kernel(const SampleArgs a, int row0, bool fill,
                                                                     RowHead* heads, const uint4* lists,
                                                                     Queue* queue, int* queued) {
  __shared__ Shared sh;
  __shared__ ListBins bins[2];
  __shared__ uint4 list[kList];
  Ctx c;
  c.sh = &sh;
  c.bins = reinterpret_cast<Bins*>(bins);
  c.x = nullptr;
  c.C = 1;
  c.rank = 0;
  const int row = row0 + blockIdx.x;
  const Settings set = settings_of(a, row);
  const float u = a.uniforms[row], s = __fdiv_rn(1.44269502f, set.T);
  const unsigned long long least =
      max(1ull, __float2ull_rn(__fmul_rn(fminf(fmaxf(set.min_p, 0.f), 1.f), kScale)));
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const RowHead head = heads[blockIdx.x];
  if (head.listed < 0) return;
  const uint4* from = lists + static_cast<size_t>(blockIdx.x) * kList;
#pragma unroll 4
  for (int i = threadIdx.x; i < head.listed; i += kThreadsB) list[i] = from[i];
  const unsigned long long cut =
      finish_row<E, kThreadsB>(c, a, set, least, u, row, list, head, s);
  if (fill && cut != ~0ull) {  // the row is -inf so far
    typename E::raw* out = static_cast<typename E::raw*>(a.filtered) + static_cast<size_t>(row) * a.V;
    for (int i = threadIdx.x; i < head.listed; i += kThreadsB) {
      const uint4 e = list[i];
      if (key_of<E>(e) <= cut && weight_of(e) >= least) {
        if constexpr (E::kBytes == 2) out[e.y] = static_cast<uint16_t>(e.x >> 16);
        else out[e.y] = __uint_as_float(e.x);
      }
    }
  }
  if (threadIdx.x == 0) {
    if (cut == ~0ull) {
      queued[atomicAdd(&queue->n, 1u)] = row;
      heads[blockIdx.x].written = 1;
    } else if (a.filtered) {
      heads[blockIdx.x].cut = cut;
    }
  }
}

// The filtered rows: 256 threads, kWriteVecs vectors each, several blocks a row.
constexpr int kWriteVecs = 8;
template <typename E>
__global__ void __launch_bounds__(256) filter_write_kernel(const SampleArgs a, int row0, int nvec, bool aligned_in,
                                                           bool aligned_out, const RowHead* heads) {
  constexpr int VEC = Staged<E>::kVec;
  const int row = row0 + blockIdx.x;
  const Settings set = settings_of(a, row);
  const float s = __fdiv_rn(1.44269502f, set.T);
  Slice<E, false> sl;
  sl.first = 0;
  sl.V = a.V;
  sl.global = static_cast<const typename E::raw*>(a.logits) + row * a.row_stride;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const RowHead head = heads[blockIdx.x];
  if (head.written) return;
  uint4 w[kWriteVecs];
#pragma unroll
  for (int i = 0; i < kWriteVecs; ++i) {
    const int v = (blockIdx.y * kWriteVecs + i) * 256 + threadIdx.x;
    if (v < nvec) w[i] = aligned_in ? ld_stream_v4(sl.global + v * VEC) : sl.at(v);
  }
  Kept kept;
  kept.cut = head.cut;
  kept.least = max(1ull, __float2ull_rn(__fmul_rn(fminf(fmaxf(set.min_p, 0.f), 1.f), kScale)));
  const float edge = head.good ? fmaxf(logit_of<E>(kept.cut), zero_logit(head.M, s)) : INFINITY;
  const bool cuts = set.k < a.V || set.min_p > 0.f || set.top_p < 1.f;
  const float sure = cuts || !head.good ? NAN : sure_logit(head.M, s);
#pragma unroll
  for (int i = 0; i < kWriteVecs; ++i) {
    const int v = (blockIdx.y * kWriteVecs + i) * 256 + threadIdx.x;
    if (v < nvec)
      write_kept<E>(a, row, 0, v, w[i], aligned_out && (v + 1) * VEC <= a.V, kept, edge, sure, head.M, s);
  }
}

// Blocks per row: the fewest whose slices fit, or 8 that read global memory.
struct Shape {
  int nvec, C, nvs;
  bool staged, split;
};
Shape shape_of(int R, int V, bool bf16) {
  Shape s;
  s.nvec = (V + (bf16 ? 8 : 4) - 1) / (bf16 ? 8 : 4);
  for (s.C = 1; s.C <= kMaxCS; s.C *= 2) {
    s.nvs = (s.nvec + s.C - 1) / s.C;
    if (s.nvs * 16ll <= (s.C == kMaxCS ? kMaxSliceS : kSliceBytesS)) {
      s.staged = true;
      s.split = static_cast<long long>(R) * s.C > kFusedBlocks;
      return s;
    }
  }
  s.C = kMaxCS;
  s.nvs = 0;
  s.staged = s.split = false;
  return s;
}

constexpr size_t kPlaceBytes = kPlaces * 2, kListBytes = kList * 16, kLongBytes = (kLongList + 1) * 16;
static_assert(sizeof(Bins) <= kPlaceBytes && 2 * sizeof(ListBins) <= sizeof(Bins) && kGroupSums * 8 <= kPlaceBytes,
              "they share the places' memory");

// Workspace: the queue, its rows, a head and a list per row.
static_assert(sizeof(Queue) <= kQueueBytes, "the queue's place");
struct Space {
  Queue* queue;
  int* queued;
  RowHead* heads;
  uint4* lists;
  size_t bytes;
};
Space space_of(void* ws, int R) {
  const size_t rows = R < kRowsAtOnce ? R : kRowsAtOnce;
  Space s;
  char* p = static_cast<char*>(ws);
  s.queue = reinterpret_cast<Queue*>(p);
  s.lists = reinterpret_cast<uint4*>(p + kQueueBytes);
  s.heads = reinterpret_cast<RowHead*>(p + kQueueBytes + rows * kListBytes);
  s.queued = reinterpret_cast<int*>(p + kQueueBytes + rows * (kListBytes + sizeof(RowHead)));
  s.bytes = (kQueueBytes + rows * (kListBytes + sizeof(RowHead) + 4) + 255) & ~static_cast<size_t>(255);
  return s;
}

template <typename E, bool kStaged>
cudaError_t launch(const SampleArgs& a, const Shape& s, const Space& sp, cudaStream_t stream) {
  const bool in = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && a.row_stride * E::kBytes % 16 == 0 &&
                  a.V % Staged<E>::kVec == 0;
  const bool out = reinterpret_cast<uintptr_t>(a.filtered) % 16 == 0 && a.V % Staged<E>::kVec == 0;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = s.C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  Queue* none = nullptr;
  // A filtered row apart from the logits is filled with -inf while they are
  // read, and what is kept added by whoever cuts; one in their place is
  // written after they have been read (filter_write_kernel).
  const char *from = static_cast<const char*>(a.logits), *to = static_cast<const char*>(a.filtered);
  const bool apart = a.filtered && (to + static_cast<size_t>(a.R) * a.V * E::kBytes <= from ||
                                    from + (static_cast<size_t>(a.R - 1) * a.row_stride + a.V) * E::kBytes <= to);
  if (!s.split) {
    cfg.gridDim = dim3(static_cast<unsigned int>(a.R) * s.C);
    cfg.blockDim = dim3(kThreadsS);
    cfg.dynamicSmemBytes = static_cast<size_t>(s.nvs) * 16 + kPlaceBytes + kListBytes;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, filter_row_kernel<E, kStaged, true>, a, 0, s.nvec, s.nvs, in, out, false, sp.heads, sp.lists,
                              kList, none, sp.queued, -0.f);
  }
  if constexpr (kStaged) {
    // blocks a row of the queue is shared by: few rows, so more than C
    int Cq = s.C;
    while (Cq < kMaxCS && s.nvec / Cq > 1024) Cq *= 2;
    const int nvq = (s.nvec + Cq - 1) / Cq;
    for (int row0 = 0; row0 < a.R; row0 += kRowsAtOnce) {
      const int rows = a.R - row0 < kRowsAtOnce ? a.R - row0 : kRowsAtOnce;
      cfg.gridDim = dim3(static_cast<unsigned int>(rows) * s.C);
      cfg.blockDim = dim3(kThreadsS);
      cfg.dynamicSmemBytes = static_cast<size_t>(s.nvs) * 16 + kPlaceBytes;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      attr[0].val.clusterDim.x = s.C;
      cudaError_t e = cudaLaunchKernelEx(&cfg, filter_row_kernel<E, true, false>, a, row0, s.nvec, s.nvs, in, out,
                                         apart, sp.heads, sp.lists, kList, sp.queue, sp.queued, -0.f);
      if (e != cudaSuccess) return e;
      // the next ones start early and wait for what they read
      cfg.gridDim = dim3(static_cast<unsigned int>(rows));
      cfg.blockDim = dim3(kThreadsB);
      cfg.dynamicSmemBytes = 0;
      cfg.attrs = attr + 1;
      e = cudaLaunchKernelEx(&cfg, filter_finish_kernel<E>, a, row0, apart, sp.heads, static_cast<const uint4*>(sp.lists),
                             sp.queue, sp.queued);
      if (e != cudaSuccess) return e;
      const int clusters = rows < kFusedBlocks / Cq ? rows : kFusedBlocks / Cq;
      cfg.gridDim = dim3(static_cast<unsigned int>(clusters * Cq));
      cfg.blockDim = dim3(kThreadsS);
      cfg.dynamicSmemBytes = static_cast<size_t>(nvq) * 16 + kPlaceBytes + kLongBytes;
      cfg.attrs = attr;
      cfg.numAttrs = 2;
      attr[0].val.clusterDim.x = Cq;
      e = cudaLaunchKernelEx(&cfg, filter_row_kernel<E, true, true>, a, row0, s.nvec, nvq, in, out, false, sp.heads, sp.lists,
                             kLongList, sp.queue, sp.queued, -0.f);
      if (e != cudaSuccess) return e;
      if (a.filtered && !apart) {
        cfg.gridDim = dim3(static_cast<unsigned int>(rows), (s.nvec + 256 * kWriteVecs - 1) / (256 * kWriteVecs));
        cfg.blockDim = dim3(256);
        cfg.dynamicSmemBytes = 0;
        cfg.attrs = attr + 1;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, filter_write_kernel<E>, a, row0, s.nvec, in, out,
                               static_cast<const RowHead*>(sp.heads));
        if (e != cudaSuccess) return e;
      }
    }
  }
  return cudaSuccess;
}

}  // namespace

size_t filtered_sample_workspace(int R, int V, bool bf16) {
  return shape_of(R, V, bf16).split ? space_of(nullptr, R).bytes : 0;
}

cudaError_t filtered_sample_prepare() {
  const int most = static_cast<int>(kMaxSliceS + kPlaceBytes + kLongBytes);
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e[] = {cudaFuncSetAttribute(filter_row_kernel<BF16, true, true>, attr, most),
                     cudaFuncSetAttribute(filter_row_kernel<F32, true, true>, attr, most),
                     cudaFuncSetAttribute(filter_row_kernel<BF16, true, false>, attr, most),
                     cudaFuncSetAttribute(filter_row_kernel<F32, true, false>, attr, most)};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

cudaError_t launch_filtered_sample(const SampleArgs& a, void* ws, cudaStream_t stream) {
  const Shape s = shape_of(a.R, a.V, a.bf16);
  const Space sp = space_of(ws, a.R);
  if (a.bf16) return s.staged ? launch<BF16, true>(a, s, sp, stream) : launch<BF16, false>(a, s, sp, stream);
  return s.staged ? launch<F32, true>(a, s, sp, stream) : launch<F32, false>(a, s, sp, stream);
}

}  // namespace specv
