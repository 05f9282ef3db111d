// filtered_sample.cu -- sampling from truncated distributions on sm_103a:
// temperature, top-k, min-p, top-p and one draw per row (the definition is in
// include/spec_decode.h).
//
// Weights are integers, w = round(2^40 * 2^t), so sums are exact in any
// order and every cut and draw is the same whatever the schedule: "the first
// element, in the order of a key, at which the running sum of weights passes
// a threshold".  The key is (descending logit, ascending index) for the cuts
// and the index for the draw.
#include <climits>

#include "device_common.cuh"
#include "launch_decode.h"
#include "sample_common.cuh"

namespace specv {
namespace {

constexpr int kThreadsS = 512;
constexpr int kWarpsS = kThreadsS / 32;

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
  if (s.T == 0.f) {
    s.T = 1.f;
    s.k = 1;
  }
  return s;
}

// Which tokens are kept: key (falling(x), index) at most (theta, last), and
// weight at least `least` (1 at the least: weight 0 is never kept).
struct Kept {
  unsigned int theta, last;
  unsigned long long least;
};

template <typename E>
struct Row {
  const void* x;
  int V;
  float M, s;
  __device__ __forceinline__ float at(int j) const { return load_one<E>(x, j); }
};

struct Shared {
  unsigned long long hist[256];
  unsigned long long sums[kWarpsS];
  float maxima[kWarpsS];
  unsigned long long rem;
  int digit;
  int any;
};

__device__ __forceinline__ unsigned long long block_sum(unsigned long long v, Shared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_sum_u64(v);
  __syncthreads();
  if (lane == 0) sh.sums[warp] = v;
  __syncthreads();
  unsigned long long t = 0;
  for (int w = 0; w < kWarpsS; ++w) t += sh.sums[w];
  return t;
}

// The lowest key at which the running sum of f(key order) passes `rem`, eight
// bits a sweep.  kBits: 54 for (falling(x), 22-bit index), 22 for the index.
// measure(j, x) is an element's weight, 0 outside the set.
template <typename E, int kBits, typename F>
__device__ unsigned long long select_key(const Row<E>& row, unsigned long long rem, F measure, Shared& sh) {
  unsigned long long prefix = 0;
  for (int top = kBits; top > 0;) {
    const int low = top > 8 ? top - 8 : 0, width = top - low;
    for (int i = threadIdx.x; i < 256; i += kThreadsS) sh.hist[i] = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < row.V; j += kThreadsS) {
      const float x = row.at(j);
      unsigned long long key = j;
      if (kBits > 22) key |= static_cast<unsigned long long>(falling(x)) << 22;
      if ((key >> top) != prefix) continue;
      const unsigned long long w = measure(j, x);
      if (w) atomicAdd(&sh.hist[(key >> low) & ((1u << width) - 1u)], w);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int d = 0, last = 0;
      unsigned long long left = rem;
      for (; d < 256; ++d) {
        if (sh.hist[d]) last = d;
        if (sh.hist[d] > left) break;
        left -= sh.hist[d];
      }
      sh.digit = d < 256 ? d : last;
      sh.rem = d < 256 ? left : 0;
    }
    __syncthreads();
    prefix = (prefix << width) | static_cast<unsigned int>(sh.digit);
    rem = sh.rem;
    top = low;
    __syncthreads();
  }
  return prefix;
}

template <typename E>
__global__ void __launch_bounds__(kThreadsS) filtered_sample_kernel(const SampleArgs a) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int r = blockIdx.x; r < a.R; r += gridDim.x) {
    const Settings set = settings_of(a, r);
    Row<E> row;
    row.x = static_cast<const char*>(a.logits) + r * a.row_stride * E::kBytes;
    row.V = a.V;
    // ---- the largest logit ----
    float M = -INFINITY;
    int odd = 0;
    for (int j = tid; j < a.V; j += kThreadsS) {
      const float x = row.at(j);
      odd |= isnan(x) || x == INFINITY;
      M = fmaxf(M, x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    __syncthreads();
    if (lane == 0) sh.maxima[warp] = M;
    odd = __syncthreads_or(odd);
    for (int w = 0; w < kWarpsS; ++w) M = fmaxf(M, sh.maxima[w]);
    const bool good = !odd && M != -INFINITY;
    row.M = M + 0.f;
    row.s = __fdiv_rn(1.44269502f, set.T);
    const float u = a.uniforms[r];
    int bad = set.bad | (good ? 0 : kDataNonfiniteLogit) | (u >= 0.f && u < 1.f ? 0 : kDataUniformRange);
    Kept kept{0xffffffffu, 0xffffffffu, 1ull};
    unsigned long long S = 0, count = 0, w_token = 0;
    int token = 0;
    if (good) {
      kept.least = max(1ull, __float2ull_rn(__fmul_rn(fminf(fmaxf(set.min_p, 0.f), 1.f), kScale)));
      auto weigh = [&](int j, float x) -> unsigned long long {
        const unsigned int key = falling(x);
        if (key > kept.theta || (key == kept.theta && static_cast<unsigned int>(j) > kept.last)) return 0;
        const unsigned long long w = weight(x, row.M, row.s);
        return w >= kept.least ? w : 0;
      };
      auto cut_at = [&](unsigned long long key) {
        kept.theta = static_cast<unsigned int>(key >> 22);
        kept.last = static_cast<unsigned int>(key & 0x3fffffu);
      };
      if (set.k < a.V)
        cut_at(select_key<E, 54>(row, set.k - 1, [](int, float) { return 1ull; }, sh));
      auto total = [&]() {
        unsigned long long t = 0, c = 0;
        for (int j = tid; j < a.V; j += kThreadsS) {
          const unsigned long long w = weigh(j, row.at(j));
          t += w;
          c += w > 0;
        }
        S = block_sum(t, sh);
        count = block_sum(c, sh);
      };
      total();
      if (set.top_p < 1.f) {
        const unsigned long long need = max(1ull, draw_threshold(fminf(fmaxf(set.top_p, 0.f), 0.99999994f), S));
        cut_at(select_key<E, 54>(row, need - 1, weigh, sh));
        total();
      }
      token = static_cast<int>(select_key<E, 22>(row, draw_threshold(u, S), weigh, sh));
      w_token = weight(row.at(token), row.M, row.s);
      if (a.filtered) {
        using raw = typename E::raw;
        const raw* src = static_cast<const raw*>(row.x);
        raw* dst = static_cast<raw*>(a.filtered) + static_cast<size_t>(r) * a.V;
        raw none;
        if constexpr (E::kBytes == 2) none = 0xff80;
        else none = -INFINITY;
        for (int j = tid; j < a.V; j += kThreadsS) dst[j] = weigh(j, row.at(j)) ? src[j] : none;
      }
    } else if (a.filtered) {
      using raw = typename E::raw;
      raw* dst = static_cast<raw*>(a.filtered) + static_cast<size_t>(r) * a.V;
      raw none;
      if constexpr (E::kBytes == 2) none = 0xff80;
      else none = -INFINITY;
      for (int j = tid; j < a.V; j += kThreadsS) dst[j] = none;
    }
    if (tid == 0) {
      a.tokens[r] = token;
      if (a.p) a.p[r] = good ? __fdiv_rn(__ull2float_rn(w_token), __ull2float_rn(S)) : 0.f;
      if (a.n_kept) a.n_kept[r] = static_cast<int>(count);
      if (bad && a.status) atomicOr(a.status, bad);
    }
    __syncthreads();
  }
}

}  // namespace

size_t filtered_sample_workspace(int R, int V, bool bf16) {
  (void)R;
  (void)V;
  (void)bf16;
  return 0;
}

cudaError_t filtered_sample_prepare() { return cudaSuccess; }

cudaError_t launch_filtered_sample(const SampleArgs& a, void* ws, int sm_count, cudaStream_t stream) {
  (void)ws;
  const int most = sm_count * 4, grid = a.R < most ? a.R : most;
  if (a.bf16) filtered_sample_kernel<BF16><<<grid, kThreadsS, 0, stream>>>(a);
  else filtered_sample_kernel<F32><<<grid, kThreadsS, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace specv
