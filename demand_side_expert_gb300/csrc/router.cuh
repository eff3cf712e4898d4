// What the two routers share: keys in the order of the floats, reductions over the
// lanes of a token, exponentials, rows in registers, sorting networks, and the
// kernel that adds the CTAs' statistics.
#pragma once

#include <math_constants.h>

#include "common.cuh"

namespace lrm {

constexpr int kRouterMaxE = 1024;
constexpr int kRouterMaxK = 32;
constexpr int kRouterMaxCtas = 160;  // partial statistics rows in the workspace

// Unsigned key in the order of the floats; -0 counts as 0 and NaN as -inf.
// Every number's key is above 0, which marks a place that was taken.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(fmaxf(x, -CUDART_INF_F) + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// Reductions over the G lanes of a token (G = 32: the warp's own instructions).
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  if constexpr (G == 32) {
    return __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = 1; o < G; o <<= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int G>
__device__ __forceinline__ uint64_t group_max(uint64_t v) {
  if constexpr (G == 32) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
    const uint32_t lo =
        __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (uint64_t)hi << 32 | lo;
  } else {
#pragma unroll
    for (int o = 1; o < G; o <<= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int G>
__device__ __forceinline__ float group_fmax(float v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// exp(x) for x <= 0 as 2^(x log2 e), on the hardware's power of two. The product's
// and the constant's rounding put the result off by up to 7e-8 |x| (1e-6 at 20 below
// the row's largest logit, 3.8e-6 at 87), and results below 2^-126 are 0. So it is used where
// that cannot be seen: in sums over a row (|x| e^x stays below 0.37), in prob_sum
// (an expert's share of which is as small as it is far down) and in gradients that
// are rounded to bfloat16. Weights and float32 gradients take expf. With expf for
// the whole row too T 32768 E 128 K 8 bfloat16, ten inputs in turn, takes 13.4 us with
// statistics instead of 12.9, and its gradient 8.7 instead of 8.1.
__device__ __forceinline__ float exp_neg(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
// The functions of a gradient in T. float32 pays for them: T 32768 E 128 K 8, ten
// inputs in turn, takes 9.3 us, 8.4 with the approximate ones.
template <typename T>
__device__ __forceinline__ float exp_grad(float x) {
  if constexpr (sizeof(T) == 4) return expf(x);
  else return exp_neg(x);
}
template <typename T>
__device__ __forceinline__ float log_grad(float x) {
  if constexpr (sizeof(T) == 4) return logf(x);
  else return __logf(x);
}
template <typename T>
__device__ __forceinline__ float inverse_grad(float x) {
  if constexpr (sizeof(T) == 4) return __frcp_rn(x);
  else return __fdividef(1.f, x);
}

// Which experts a lane holds: chunks of kVec consecutive ones (16 bytes at
// most), the chunks of the G lanes side by side: expert of slot i of lane l is
// (i / kVec * G + l) * kVec + i % kVec.
template <typename T, int NI, int G>
struct RowShape {
  static constexpr int kVec = NI * (int)sizeof(T) < 16 ? NI : 16 / (int)sizeof(T);
  __device__ __forceinline__ static int expert(int i, int lane) {
    return (i / kVec * G + lane) * kVec + i % kVec;
  }
};

template <int BYTES>
__device__ __forceinline__ void copy_bytes(void* dst, const void* src) {
  if constexpr (BYTES == 16) *(uint4*)dst = *(const uint4*)src;
  else if constexpr (BYTES == 8) *(uint2*)dst = *(const uint2*)src;
  else if constexpr (BYTES == 4) *(uint32_t*)dst = *(const uint32_t*)src;
  else *(uint16_t*)dst = *(const uint16_t*)src;
}

// The lane's logits, -inf past E. vec: rows begin on a multiple of a chunk, so
// a chunk wholly inside the row is one load.
template <typename T, int NI, int G>
__device__ __forceinline__ void load_row(const T* row, int lane, int E, bool vec, float (&x)[NI]) {
  using S = RowShape<T, NI, G>;
#pragma unroll
  for (int c = 0; c < NI / S::kVec; ++c) {
    const int e = S::expert(c * S::kVec, lane);
    alignas(16) T v[S::kVec];
    if (vec && e + S::kVec <= E) {
      copy_bytes<S::kVec * (int)sizeof(T)>(v, row + e);
#pragma unroll
      for (int i = 0; i < S::kVec; ++i) x[c * S::kVec + i] = (float)v[i];
    } else {
#pragma unroll
      for (int i = 0; i < S::kVec; ++i)
        x[c * S::kVec + i] = e + i < E ? (float)row[e + i] : -CUDART_INF_F;
    }
  }
}

// Minima and maxima on registers: sorted lists of 32-bit keys, largest first.
__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b), lo = min(a, b);
  a = hi;
  b = lo;
}
// Sorts v[0 .. N) descending (odd-even merge sort; N a power of two up to 8).
template <int N>
__device__ __forceinline__ void sort_desc(uint32_t* v) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p))
            exchange(v[i + j], v[i + j + k]);
}
// Sorts a bitonic sequence descending.
template <int N>
__device__ __forceinline__ void merge_desc(uint32_t* v) {
#pragma unroll
  for (int s = N / 2; s >= 1; s /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & s) == 0) exchange(v[i], v[i + s]);
}
// a := the N largest of two descending lists of N, descending.
template <int N>
__device__ __forceinline__ void top_of(uint32_t* a, const uint32_t* b) {
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = max(a[i], b[N - 1 - i]);
  merge_desc<N>(a);
}
// L sorted keys of this lane and of the lanes 1, 2, .. G / 2 away, KC kept.
template <int G, int KC, int L, int O>
__device__ __forceinline__ void merge_lanes(uint32_t (&v)[KC]) {
  if constexpr (O < G) {
    if constexpr (L < KC) {
#pragma unroll
      for (int i = 0; i < L; ++i) v[2 * L - 1 - i] = __shfl_xor_sync(0xffffffffu, v[i], O);
      merge_desc<2 * L>(v);
      merge_lanes<G, KC, 2 * L, 2 * O>(v);
    } else {
      uint32_t u[KC];
#pragma unroll
      for (int i = 0; i < KC; ++i) u[i] = __shfl_xor_sync(0xffffffffu, v[i], O);
      top_of<KC>(v, u);
      merge_lanes<G, KC, KC, 2 * O>(v);
    }
  }
}

// Adds the routing CTAs' sums in a fixed order and forms the losses: one cluster,
// every CTA an eighth of the experts, 32 experts at a time (a lane each) by 16
// shares of the rows (a warp each); the CTAs' parts of the loss meet in the first
// one's shared memory. 2 us at E 128, launch included.
constexpr int kSumCtas = 8, kSumThreads = 512, kSumWarps = kSumThreads / 32;
static_assert(kRouterMaxCtas % 32 == 0, "whole shares");
static __global__ void __cluster_dims__(kSumCtas, 1, 1) __launch_bounds__(kSumThreads)
route_sums_kernel(const float2* __restrict__ part, const float* __restrict__ part_z, int rows,
                  int E, int K, float balance_coef, float z_coef, int32_t* __restrict__ counts,
                  float* __restrict__ prob_sum, float* __restrict__ loss) {
  constexpr int kWarps = kSumWarps;
  __shared__ float2 sm[2][kWarps][33];
  __shared__ float2 red[kWarps];
  __shared__ float2 all[kSumCtas];  // (sum of counts P, sum of counts) of every CTA
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)cluster_ctarank();
  const int per = (E + kSumCtas - 1) / kSumCtas;
  const int begin = rank * per, end = min(E, begin + per);
  // every CTA has started before another writes to its shared memory; waited for below
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  pdl_begin();  // predecessor complete before any global access
  float z = 0.f;
  if (rank == 0 && warp == 0 && part_z) {
#pragma unroll
    for (int k = 0; k < kRouterMaxCtas / 32; ++k)
      z += lane + 32 * k < rows ? part_z[lane + 32 * k] : 0.f;
  }
  float dot = 0.f, cnt = 0.f;
  int buf = 0;
  for (int e0 = begin; e0 < end; e0 += 32, buf ^= 1) {
    // every load before any use
    float2 v[kRouterMaxCtas / kWarps];
#pragma unroll
    for (int k = 0; k < kRouterMaxCtas / kWarps; ++k) {
      const int r = warp + k * kWarps;
      v[k] = e0 + lane < end && r < rows ? part[(int64_t)r * E + e0 + lane]
                                         : make_float2(0.f, 0.f);
    }
    float s = 0.f;
    int c = 0;
#pragma unroll
    for (int k = 0; k < kRouterMaxCtas / kWarps; ++k) {
      s += v[k].x;
      c += __float_as_int(v[k].y);
    }
    sm[buf][warp][lane] = make_float2(s, __int_as_float(c));
    __syncthreads();
    // warp w adds experts 2 w and 2 w + 1, half a warp each
    const int col = 2 * warp + lane / 16;
    const float2 u = sm[buf][lane % 16][col];
    s = u.x;
    c = __float_as_int(u.y);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      c += __shfl_xor_sync(0xffffffffu, c, o);
    }
    const int e = e0 + col;
    if (lane % 16 == 0 && e < end) {
      prob_sum[e] = s;
      counts[e] = c;
      dot = fmaf((float)c, s, dot);
      cnt += (float)c;
    }
  }
  dot = warp_sum(dot);
  cnt = warp_sum(cnt);
  if (lane == 0) red[warp] = make_float2(dot, cnt);
  __syncthreads();
  asm volatile("barrier.cluster.wait;" ::: "memory");
  if (warp == 0) {
    dot = warp_sum(lane < kWarps ? red[lane].x : 0.f);
    cnt = warp_sum(lane < kWarps ? red[lane].y : 0.f);
    z = warp_sum(z);
    if (lane == 0) {
      const uint32_t mine = (uint32_t)__cvta_generic_to_shared(&all[rank]);
      uint32_t first;
      asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(first) : "r"(mine));
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(first), "f"(dot), "f"(cnt)
                   : "memory");
    }
  }
  cluster_barrier();  // every CTA's part has arrived in the first one
  if (rank == 0 && warp == 0) {
    const float d = warp_sum(lane < kSumCtas ? all[lane].x : 0.f);
    // tokens that took part: every one chose K experts
    const float n = fmaxf(warp_sum(lane < kSumCtas ? all[lane].y : 0.f) / (float)K, 1.f);
    if (lane == 0) {
      loss[0] = balance_coef * (float)E * (d / (n * n * (float)K));
      if (part_z) loss[1] = z_coef * (z / n);  // a router without a z-loss has none
    }
  }
}

inline lrm_status check_aligned(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return LRM_ERR_UNSUPPORTED;
  return LRM_OK;
}

}  // namespace lrm
