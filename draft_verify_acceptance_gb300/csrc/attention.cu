// attention.cu -- attention of the newest Q tokens of each sequence over its
// paged keys and values (sm_103a).
//
//   s_rt = scale * q_r . k_t,  out_r = sum_t e^(s_rt - m_r) v_t / l_r,
//   l_r = sum_t e^(s_rt - m_r),  m_r a running maximum,
// for the tokens t <= n - Q + i that query i of a sequence of n tokens sees.
#include "attention_common.cuh"
#include "attention_mma.cuh"

namespace specv {
namespace {

// ---- fp32 multiply-adds ----------------------------------------------------
constexpr int kRowsF = 8;       // rows an item holds
constexpr int kWarpsF = 4;
constexpr int kThreadsF = kWarpsF * 32;
constexpr int kStepF = kThreadsF;  // tokens a CTA takes per step: one a thread

// Element type loads of 4 consecutive values.
template <typename E>
__device__ __forceinline__ float4 load4(const char* p) {
  if constexpr (E::kBytes == 4) {
    return __ldg(reinterpret_cast<const float4*>(p));
  } else {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
  }
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreadsF) attention_kernel(const AttnArgs a) {
  constexpr int DL = D / 32;  // dimensions a lane accumulates
  __shared__ __align__(16) float s_q[kRowsF][D];
  __shared__ __align__(16) float s_p[kWarpsF][kRowsF][32];
  __shared__ const char* s_v[kWarpsF][32];
  __shared__ __align__(16) float s_o[kWarpsF][kRowsF][D];
  __shared__ float s_m[kWarpsF][kRowsF], s_l[kWarpsF][kRowsF];
  __shared__ long long s_plan[2 * kWarpsF + 4];
  __shared__ int s_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = a.cache.heads, G = a.Hq / H, R = a.Q * G;
  const int RT = (R + kRowsF - 1) / kRowsF;
  const int S = a.cache.page_size;
  AttnPlan plan = attn_plan<kStepF, kThreadsF>(a, H * RT, 1, s_plan);
  long long w = plan.per * blockIdx.x;
  const long long end = min(plan.total, w + plan.per);
  int b = plan.b;
  long long base = plan.base;
  while (w < end) {
    int n = attn_length(a, b), tiles = attn_tiles<kStepF>(n);
    while (w >= base + static_cast<long long>(tiles) * H * RT) {
      base += static_cast<long long>(tiles) * H * RT;
      n = attn_length(a, ++b);
      tiles = attn_tiles<kStepF>(n);
    }
    const int item = static_cast<int>((w - base) / tiles);
    const int tile0 = static_cast<int>((w - base) - static_cast<long long>(item) * tiles);
    const int tile1 = static_cast<int>(min(static_cast<long long>(tiles), tile0 + (end - w)));
    const int rt = item / H, h = item - rt * H;
    const int row0 = rt * kRowsF, rows = min(kRowsF, R - row0);
    const int32_t* table = a.table.ids + b * a.table.stride;

    __syncthreads();
    for (int e = tid; e < kRowsF * (D / 4); e += kThreadsF) {
      const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        const AttnRow ar = attn_row(a, row0 + r, h);
        v = load4<E>(a.q + b * a.q_batch + ar.i * a.q_token + ar.hq * a.q_head + d * E::kBytes);
      }
      *reinterpret_cast<float4*>(&s_q[r][d]) = v;
    }
    __syncthreads();
    float m[kRowsF], l[kRowsF], o[kRowsF][DL];
#pragma unroll
    for (int r = 0; r < kRowsF; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int k = 0; k < DL; ++k) o[r][k] = 0.f;
    }
    for (int tile = tile0; tile < tile1; ++tile) {
      const int t0 = tile * kStepF + warp * 32, t = t0 + lane;
      const int count = min(32, n - t0);
      if (count <= 0) continue;
      float s[kRowsF];
      long long off = -1;
      if (t < n) {
        const int page = table[t / S];
        if (page >= 0 && page < a.cache.pages)
          off = page * a.cache.page_stride + (t % S) * a.cache.token_stride + h * (D * E::kBytes);
        else if (a.status)
          atomicOr(a.status, kDataPageRange);
      }
      s_v[warp][lane] = off < 0 ? nullptr : a.cache.v + off;
#pragma unroll
      for (int r = 0; r < kRowsF; ++r) s[r] = 0.f;
      if (off >= 0) {
        for (int d = 0; d < D; d += 4) {
          const float4 k = load4<E>(a.cache.k + off + d * E::kBytes);
#pragma unroll
          for (int r = 0; r < kRowsF; ++r) {
            const float4 q = *reinterpret_cast<const float4*>(&s_q[r][d]);
            s[r] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[r]))));
          }
        }
      }
#pragma unroll
      for (int r = 0; r < kRowsF; ++r) {
        const int i = (row0 + r) / G;
        const bool seen = off >= 0 && r < rows && t <= n - a.Q + i;
        s[r] = seen ? s[r] * a.scale_log2 : -INFINITY;
        float mx = s[r];
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        const float mn = fmaxf(m[r], mx);
        const float c = m[r] == -INFINITY ? 0.f : ex2(m[r] - mn);
        const float p = seen ? ex2(s[r] - mn) : 0.f;
        l[r] = fmaf(l[r], c, p);
#pragma unroll
        for (int k = 0; k < DL; ++k) o[r][k] *= c;
        m[r] = mn;
        // a token that the row does not see is marked, and not multiplied
        s_p[warp][r][lane] = seen ? p : -1.f;
      }
      __syncwarp();
      for (int j = 0; j < count; ++j) {
        const char* vp = s_v[warp][j];
        if (!vp) continue;
        float v[DL];
#pragma unroll
        for (int k = 0; k < DL; k += 2) {
          if constexpr (E::kBytes == 4) {
            const float2 x = __ldg(reinterpret_cast<const float2*>(vp + (lane * DL + k) * 4));
            v[k] = x.x;
            v[k + 1] = x.y;
          } else {
            const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(vp + (lane * DL + k) * 2));
            v[k] = bf16_lo(x);
            v[k + 1] = bf16_hi(x);
          }
        }
#pragma unroll
        for (int r = 0; r < kRowsF; ++r) {
          const float p = s_p[warp][r][j];
          if (p >= 0.f) {
#pragma unroll
            for (int k = 0; k < DL; ++k) o[r][k] = fmaf(p, v[k], o[r][k]);
          }
        }
      }
      __syncwarp();
    }
    // ---- the warps' parts, then the item's ----
#pragma unroll
    for (int r = 0; r < kRowsF; ++r) {
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
      if (lane == 0) {
        s_m[warp][r] = m[r];
        s_l[warp][r] = l[r];
      }
#pragma unroll
      for (int k = 0; k < DL; ++k) s_o[warp][r][lane * DL + k] = o[r][k];
    }
    __syncthreads();
    const bool whole = tile0 == 0 && tile1 == tiles;
    float* slot = attn_slot<kRowsF, D>(a, blockIdx.x, tile0 == 0);
    for (int e = tid; e < rows * (D / 4); e += kThreadsF) {
      const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
      float mm = -INFINITY, ll = 0.f;
      float4 oo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < kWarpsF; ++x) mm = fmaxf(mm, s_m[x][r]);
#pragma unroll
      for (int x = 0; x < kWarpsF; ++x) {
        const float c = s_m[x][r] == -INFINITY ? 0.f : ex2(s_m[x][r] - mm);
        const float4 v = *reinterpret_cast<const float4*>(&s_o[x][r][d]);
        ll = fmaf(c, s_l[x][r], ll);
        oo.x = fmaf(c, v.x, oo.x);
        oo.y = fmaf(c, v.y, oo.y);
        oo.z = fmaf(c, v.z, oo.z);
        oo.w = fmaf(c, v.w, oo.w);
      }
      if (whole) {
        attn_write<D>(a, b, h, row0 + r, d, mm, ll, oo);
      } else {
        *reinterpret_cast<float4*>(slot + r * D + d) = oo;
        if (d == 0) {
          slot[kRowsF * D + r] = mm;
          slot[kRowsF * D + kRowsF + r] = ll;
        }
      }
    }
    if (!whole) {
      const long long first = base + static_cast<long long>(item) * tiles;
      if (attn_arrive(a, first, tiles, plan.per, &s_flag))
        attn_join<kRowsF, D, kThreadsF>(a, b, h, row0, rows, first, tiles, plan.per);
    }
    w += tile1 - tile0;
  }
}

}  // namespace

// Rows a cache head (R = Q * Hq / Hkv) choose the bf16 kernel: up to 24 go to
// attention_mma.cuh, more to attention_tc.cuh.  At 64 sequences of 400..4000
// tokens, Hq 32, Hkv 8, D 128 (floor 94 to 96 us) the two took
//   R = 4: 109 and 147 us;  16: 126 and 147;  24: 140 and 178;
//   R = 32: 235 and 180;    68: 360 and 302
// (a fourth block of 8 rows leaves mma without registers; its K and V come
// through L2 once more a block of rows), with D 64 and R = 24: 100 and 149.
constexpr int kMmaRows = 24;
constexpr int kMaxMmaCtas = 304;

size_t attention_workspace(int D, bool bf16) {
  const size_t rows = bf16 ? kMaxRowsTc : kRowsF;
  const size_t ctas = bf16 ? kMaxMmaCtas : kAttnMaxCtas;
  return (static_cast<size_t>(kAttnMaxCtas) * 4 + ctas * 2 * rows * (D + 2) * 4 + 255) & ~static_cast<size_t>(255);
}

cudaError_t attention_prepare() {
  cudaError_t e[] = {mma::prepare<64, 1>(),  mma::prepare<64, 2>(),  mma::prepare<64, 3>(),
                     mma::prepare<128, 1>(), mma::prepare<128, 2>(), mma::prepare<128, 3>(),
                     attention_tc_prepare_64(), attention_tc_prepare_128()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

cudaError_t launch_attention(const AttnArgs& a, int sm_count, cudaStream_t stream) {
  const bool wide = a.cache.head_dim == 128;
  if (!a.cache.bf16) {
    const int grid = sm_count * 3 < kAttnMaxCtas ? sm_count * 3 : kAttnMaxCtas;
    if (wide) attention_kernel<F32, 128><<<grid, kThreadsF, 0, stream>>>(a);
    else attention_kernel<F32, 64><<<grid, kThreadsF, 0, stream>>>(a);
    return cudaGetLastError();
  }
  const int R = a.Q * (a.Hq / a.cache.heads);
  if (R <= kMmaRows) {
    const int grid = sm_count * 2 < kMaxMmaCtas ? sm_count * 2 : kMaxMmaCtas;
    switch ((R + 7) / 8 + (wide ? 3 : 0)) {
      case 1: mma::launch<64, 1>(a, grid, stream); break;
      case 2: mma::launch<64, 2>(a, grid, stream); break;
      case 3: mma::launch<64, 3>(a, grid, stream); break;
      case 4: mma::launch<128, 1>(a, grid, stream); break;
      case 5: mma::launch<128, 2>(a, grid, stream); break;
      default: mma::launch<128, 3>(a, grid, stream); break;
    }
    return cudaGetLastError();
  }
  // rows in tiles of equal size, a multiple of 16 and at most 96 (and so 32 at least)
  const int tiles = (R + kMaxRowsTc - 1) / kMaxRowsTc;
  const int n16 = ((R + tiles - 1) / tiles + 15) / 16;
  const int grid = sm_count < kMaxMmaCtas ? sm_count : kMaxMmaCtas;
  if (wide) attention_tc_launch_128(a, n16, grid, stream);
  else attention_tc_launch_64(a, n16, grid, stream);
  return cudaGetLastError();
}

}  // namespace specv
