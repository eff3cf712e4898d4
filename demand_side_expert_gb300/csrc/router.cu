// Router of the MoE layer: top-K experts of every token with their routing
// weights, per-expert counts, the balance loss and the z-loss, and the
// gradient of all of them with respect to the logits.
//
// For the tokens t that take part (mask, and at least one logit above -inf):
//   p_t = softmax(x_t),  lse_t = log sum_e exp(x_te)
//   I_t = the K largest logits, ties to the lower expert id
//   alpha_tk = p at I_t (renorm: divided by its sum over I_t)
//   counts_e = #{(t, k): I_tk = e},  P_e = sum_t p_te,  n = #tokens
//   balance = c_b E / (n^2 K) sum_e counts_e P_e,   z = c_z / n sum_t lse_t^2
// counts are constants to the gradient (they are piecewise constant).
//
// A warp per token: lane l holds the NI consecutive experts l*NI .. of the
// row in registers, so a row is read once, the lowest lane of a tie is the
// lowest expert, and no shared memory is touched before the statistics.
#include <math_constants.h>

#include <algorithm>

#include "common.cuh"

namespace lrm {

constexpr int kRouterMaxE = 1024;
constexpr int kRouterMaxK = 32;
constexpr int kRouterMaxCtas = 160;  // partial statistics rows in the workspace

// The statistics' ticket is word 1 of the workspace header.
inline uint32_t* router_ticket(void* ws) { return static_cast<uint32_t*>(ws) + 1; }

// Unsigned key in the order of the floats; -0 counts as 0 and NaN as -inf.
// Every number's key is above 0, which marks "taken" or "no such expert".
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) x = -CUDART_INF_F;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) {
  return __bfloat162float(*p);
}
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16_rn(v);
}

template <typename T, int NI>
__device__ __forceinline__ void load_row(const T* row, int e0, int E, float (&x)[NI]) {
#pragma unroll
  for (int i = 0; i < NI; ++i) x[i] = e0 + i < E ? load_logit(row + e0 + i) : -CUDART_INF_F;
}

// Whether token t takes part: its row maximum is above -inf, or it holds a
// NaN (which then reaches the outputs), and it is not masked out.
template <int NI>
__device__ __forceinline__ bool takes_part(const float (&x)[NI], float top, const uint8_t* mask,
                                           int64_t t) {
  if (mask && mask[t] == 0) return false;
  if (top > -CUDART_INF_F) return true;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NI; ++i) nan |= x[i] != x[i];
  return __any_sync(0xffffffffu, nan);
}

template <typename T, int NI, bool STATS>
__global__ void __launch_bounds__(1024)
route_kernel(const T* __restrict__ logits, const uint8_t* __restrict__ mask, int ntok, int E,
             int K, int64_t stride, int renorm, float balance_coef, float z_coef,
             int32_t* __restrict__ topk_idx, float* __restrict__ alpha,
             int32_t* __restrict__ counts, float* __restrict__ prob_sum,
             float* __restrict__ loss, float* part_p, int32_t* part_c, float* part_z,
             uint32_t* ticket) {
  pdl_begin();  // predecessor complete before any global access
  extern __shared__ float sm[];  // STATS: [warps][E] sums of p, then [E] counts, [warps] lse^2
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarp = blockDim.x >> 5;
  const int e0 = lane * NI;
  float* sm_p = sm;
  int32_t* sm_c = reinterpret_cast<int32_t*>(sm + (int64_t)nwarp * E);
  float* sm_z = reinterpret_cast<float*>(sm_c + E);
  float acc[NI];
  float zacc = 0.f;
  if constexpr (STATS) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) sm_c[e] = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) acc[i] = 0.f;
    __syncthreads();
  }
  for (int64_t t = (int64_t)blockIdx.x * nwarp + warp; t < ntok; t += (int64_t)gridDim.x * nwarp) {
    float x[NI];
    uint32_t key[NI];
    load_row<T, NI>(logits + t * stride, e0, E, x);
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      key[i] = e0 + i < E ? order_key(x[i]) : 0u;
      if (key[i] > best) { best = key[i]; at = i; }
    }
    // lane k keeps the k-th choice
    uint32_t my_key = 0, top_key = 0;
    int my_idx = 0;
    for (int k = 0; k < K; ++k) {
      const uint32_t hi = __reduce_max_sync(0xffffffffu, best);
      const int src = __ffs(__ballot_sync(0xffffffffu, best == hi)) - 1;
      const int idx = __shfl_sync(0xffffffffu, e0 + at, src);
      if (k == 0) top_key = hi;
      if (lane == k) { my_key = hi; my_idx = idx; }
      if (lane == src) {
        best = 0;
        const int gone = at;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (i == gone) key[i] = 0;
          if (key[i] > best) { best = key[i]; at = i; }
        }
      }
    }
    const float top = key_value(top_key);
    const bool use = takes_part(x, top, mask, t);
    // p, its sum over the row, and the weights of the K choices
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      x[i] = expf(x[i] - top);  // 0 past E: -inf - top
      if (e0 + i >= E) x[i] = 0.f;
      total += x[i];
    }
    total = warp_sum(total);
    float a = lane < K ? expf(key_value(my_key) - top) : 0.f;
    const float den = renorm ? warp_sum(a) : total;
    // a NaN in the row makes every weight NaN, also where the choices' own sum has none
    a = total != total ? total : a / den;
    if (lane < K) {
      topk_idx[t * K + lane] = my_idx;
      alpha[t * K + lane] = use ? a : 0.f;
    }
    if constexpr (STATS) {
      if (use) {
        const float inv_total = 1.f / total;
#pragma unroll
        for (int i = 0; i < NI; ++i) acc[i] = fmaf(x[i], inv_total, acc[i]);
        const float lse = top + logf(total);
        zacc = fmaf(lse, lse, zacc);
        if (lane < K) atomicAdd(&sm_c[my_idx], 1);
      }
    }
  }
  if constexpr (STATS) {
    // CTA sums in a fixed order; then the last CTA to arrive adds the CTAs'
    // sums, in CTA order: the result does not depend on the arrival order
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (e0 + i < E) sm_p[(int64_t)warp * E + e0 + i] = acc[i];
    if (lane == 0) sm_z[warp] = zacc;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      float s = 0.f;
      for (int w = 0; w < nwarp; ++w) s += sm_p[(int64_t)w * E + e];
      part_p[(int64_t)blockIdx.x * E + e] = s;
      part_c[(int64_t)blockIdx.x * E + e] = sm_c[e];
    }
    if (threadIdx.x == 0) {
      float s = 0.f;
      for (int w = 0; w < nwarp; ++w) s += sm_z[w];
      part_z[blockIdx.x] = s;
    }
    __shared__ bool last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicInc(ticket, gridDim.x - 1) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    float dot = 0.f, cnt = 0.f;
    __shared__ float red[2][32];
    int64_t pairs = 0;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      float s = 0.f;
      int32_t c = 0;
      for (int b = 0; b < (int)gridDim.x; ++b) {
        s += __ldcg(part_p + (int64_t)b * E + e);
        c += __ldcg(part_c + (int64_t)b * E + e);
      }
      prob_sum[e] = s;
      counts[e] = c;
      dot = fmaf((float)c, s, dot);
      pairs += c;
    }
    // tokens that took part: every one chose K experts
    cnt = (float)pairs;
    dot = warp_sum(dot);
    cnt = warp_sum(cnt);
    if (lane == 0) { red[0][warp] = dot; red[1][warp] = cnt; }
    __syncthreads();
    if (threadIdx.x == 0) {
      float d = 0.f, n = 0.f, z = 0.f;
      for (int w = 0; w < nwarp; ++w) { d += red[0][w]; n += red[1][w]; }
      for (int b = 0; b < (int)gridDim.x; ++b) z += __ldcg(part_z + b);
      n = fmaxf(n / (float)K, 1.f);
      loss[0] = balance_coef * (float)E * (d / (n * n * (float)K));
      loss[1] = z_coef * (z / n);
    }
  }
}

template <typename T, int NI>
__global__ void __launch_bounds__(256)
route_bwd_kernel(const T* __restrict__ logits, const uint8_t* __restrict__ mask,
                 const int32_t* __restrict__ topk_idx, const int32_t* __restrict__ counts,
                 const float* __restrict__ dalpha, const float* __restrict__ dloss, int ntok,
                 int E, int K, int64_t stride, int renorm, float balance_coef, float z_coef,
                 T* __restrict__ dlogits, int32_t* err) {
  pdl_begin();  // predecessor complete before any global access
  const int lane = threadIdx.x & 31;
  const int e0 = lane * NI;
  // d balance / d p_te of the lane's experts, and 2 c_z / n of the z-loss
  float cost[NI];
  int64_t pairs = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int c = e0 + i < E ? counts[e0 + i] : 0;
    pairs += c;
    cost[i] = (float)c;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) pairs += __shfl_xor_sync(0xffffffffu, pairs, o);
  const float n = fmaxf((float)pairs / (float)K, 1.f);
  const float d0 = dloss ? dloss[0] : 1.f, d1 = dloss ? dloss[1] : 1.f;
  const float kb = d0 * balance_coef * (float)E / (n * n * (float)K);
  const float kz = d1 * 2.f * z_coef / n;
#pragma unroll
  for (int i = 0; i < NI; ++i) cost[i] *= kb;

  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t t = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; t < ntok; t += nwarps) {
    float x[NI], d[NI];
    load_row<T, NI>(logits + t * stride, e0, E, x);
    uint32_t hi = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) hi = max(hi, e0 + i < E ? order_key(x[i]) : 0u);
    const float top = key_value(__reduce_max_sync(0xffffffffu, hi));
    const bool use = takes_part(x, top, mask, t);
    int my_idx = -1;
    float my_da = 0.f;
    if (lane < K) {
      const int q = topk_idx[t * K + lane];
      if (q >= 0 && q < E) my_idx = q;
      else flag_error(err, LRM_DEVERR_EXPERT_ID);
      if (dalpha && my_idx >= 0) my_da = dalpha[t * K + lane];
    }
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      x[i] = e0 + i < E ? expf(x[i] - top) : 0.f;
      d[i] = 0.f;
      total += x[i];
    }
    total = warp_sum(total);
    const float inv_total = 1.f / total;
    // the lane of choice k gets dalpha_k at its expert
    float my_ex = 0.f;  // exp(x - top) of the lane's own choice
    for (int k = 0; k < K; ++k) {
      const int idx = __shfl_sync(0xffffffffu, my_idx, k);
      const float da = __shfl_sync(0xffffffffu, my_da, k);
      const int owner = idx < 0 ? 0 : idx / NI;
      float ex = 0.f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (e0 + i == idx) { d[i] = da; ex = x[i]; }
      ex = __shfl_sync(0xffffffffu, ex, owner);
      if (lane == k && idx >= 0) my_ex = ex;
    }
    // sum over the choices of alpha dalpha (renorm), or of p dalpha
    const float den = renorm ? warp_sum(my_ex) : total;
    const float mean = warp_sum(my_ex * my_da) / den;
    float cmean = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) cmean = fmaf(x[i] * inv_total, cost[i], cmean);
    cmean = warp_sum(cmean);
    const float zterm = kz * (top + logf(total));
    // lanes whose experts were chosen: under renorm only they see dalpha
    uint32_t chosen = 0;
    if (renorm) {
      for (int k = 0; k < K; ++k) {
        const int idx = __shfl_sync(0xffffffffu, my_idx, k);
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (e0 + i == idx) chosen |= 1u << i;
      }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (e0 + i >= E) continue;
      const float p = x[i] * inv_total;
      float v = p * (cost[i] - cmean + zterm);
      if (renorm) {
        if (chosen >> i & 1) v = fmaf(x[i] / den, d[i] - mean, v);
      } else {
        v = fmaf(p, d[i] - mean, v);
      }
      store_logit(dlogits + t * E + e0 + i, use ? v : 0.f);
    }
  }
}

static lrm_status check_router(const lrm_router* r) {
  if (!r) return LRM_ERR_INVALID_ARG;
  if (r->T < 0 || r->E <= 0 || r->K <= 0 || r->K > r->E) return LRM_ERR_INVALID_ARG;
  if (r->dtype != LRM_F32 && r->dtype != LRM_BF16) return LRM_ERR_INVALID_ARG;
  if (r->stride < r->E) return LRM_ERR_INVALID_ARG;
  if (r->E > kRouterMaxE || r->K > kRouterMaxK) return LRM_ERR_UNSUPPORTED;
  if ((int64_t)r->T * r->K >= (int64_t)1 << 31) return LRM_ERR_UNSUPPORTED;
  return LRM_OK;
}

static size_t router_bytes(const lrm_router* r) {
  // header, then sums of p, counts and lse^2 of every CTA
  const size_t b = kWsHeaderBytes + (size_t)kRouterMaxCtas * (8 * (size_t)r->E + 4);
  return (b + 255) / 256 * 256;
}

static lrm_status check_router_ws(const lrm_router* r, const void* ws, size_t ws_bytes) {
  if (!ws) return LRM_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return LRM_ERR_UNSUPPORTED;
  if (ws_bytes < router_bytes(r)) return LRM_ERR_WORKSPACE;
  return LRM_OK;
}

static lrm_status check_aligned(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return LRM_ERR_UNSUPPORTED;
  return LRM_OK;
}

template <typename T, int NI>
static lrm_status launch_route(const lrm_router* r, const void* logits, const uint8_t* mask,
                               int32_t* topk_idx, float* alpha, int32_t* counts,
                               float* prob_sum, float* loss, void* ws, cudaStream_t cs) {
  const bool stats = counts != nullptr;
  // as many warps as tokens up to 32 a CTA and one CTA an SM, the rounds even
  const int max_warps = NI >= 32 ? 16 : 32;
  const int64_t ctas = std::min(num_sms(), kRouterMaxCtas);
  const int64_t rounds = std::max<int64_t>(1, (r->T + ctas * max_warps - 1) / (ctas * max_warps));
  const int64_t need = std::max<int64_t>(1, (r->T + rounds - 1) / rounds);
  const int nwarp = (int)std::min<int64_t>(max_warps, need);
  const int grid = (int)((need + nwarp - 1) / nwarp);
  float* part_p = reinterpret_cast<float*>((char*)ws + kWsHeaderBytes);
  int32_t* part_c = reinterpret_cast<int32_t*>(part_p + (size_t)kRouterMaxCtas * r->E);
  float* part_z = reinterpret_cast<float*>(part_c + (size_t)kRouterMaxCtas * r->E);
  auto kern = stats ? route_kernel<T, NI, true> : route_kernel<T, NI, false>;
  const size_t smem = stats ? ((size_t)nwarp * r->E + r->E + nwarp) * 4 : 0;
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
          cudaSuccess)
    return LRM_ERR_CUDA;
  if (launch_k(kern, dim3(grid), dim3(nwarp * 32), smem, cs, (const T*)logits, mask, r->T, r->E,
               r->K, r->stride, r->renorm, r->balance_coef, r->z_coef, topk_idx, alpha, counts,
               prob_sum, loss, part_p, part_c, part_z, router_ticket(ws)) != cudaSuccess) {
    (void)cudaGetLastError();
    return LRM_ERR_CUDA;
  }
  return launch_status();
}

template <typename T, int NI>
static lrm_status launch_route_bwd(const lrm_router* r, const void* logits, const uint8_t* mask,
                                   const int32_t* topk_idx, const int32_t* counts,
                                   const float* dalpha, const float* dloss, void* dlogits,
                                   int32_t* err, cudaStream_t cs) {
  const int64_t blocks = std::min<int64_t>(((int64_t)r->T + 7) / 8, (int64_t)num_sms() * 8);
  launch_k(route_bwd_kernel<T, NI>, dim3((unsigned)blocks), dim3(256), 0, cs, (const T*)logits,
           mask, topk_idx, counts, dalpha, dloss, r->T, r->E, r->K, r->stride, r->renorm,
           r->balance_coef, r->z_coef, (T*)dlogits, err);
  return launch_status();
}

// Experts a lane: the smallest power of two that covers E with 32 lanes.
#define LRM_ROUTER_NI(call, T)            \
  (r->E <= 32    ? call<T, 1>             \
   : r->E <= 64  ? call<T, 2>             \
   : r->E <= 128 ? call<T, 4>             \
   : r->E <= 256 ? call<T, 8>             \
   : r->E <= 512 ? call<T, 16>            \
                 : call<T, 32>)

}  // namespace lrm

using namespace lrm;

extern "C" size_t lrm_router_workspace_bytes(const lrm_router* r) {
  return check_router(r) == LRM_OK ? router_bytes(r) : 0;
}

extern "C" lrm_status lrm_route(const lrm_router* r, const void* logits, const uint8_t* mask,
                                int32_t* topk_idx, float* alpha, int32_t* counts,
                                float* prob_sum, float* loss, void* ws, size_t ws_bytes,
                                void* stream) {
  LRM_NVTX("lrm_route");
  lrm_status st = check_router(r);
  if (st != LRM_OK) return st;
  if ((st = check_router_ws(r, ws, ws_bytes)) != LRM_OK) return st;
  const int given = !!counts + !!prob_sum + !!loss;
  if (given != 0 && given != 3) return LRM_ERR_INVALID_ARG;
  if (r->T > 0 && (!logits || !topk_idx || !alpha)) return LRM_ERR_INVALID_ARG;
  if ((st = check_aligned({logits, topk_idx, alpha, counts, prob_sum, loss})) != LRM_OK)
    return st;
  if (r->T == 0 && !counts) return LRM_OK;
  cudaStream_t cs = (cudaStream_t)stream;
  auto go = r->dtype == LRM_BF16 ? LRM_ROUTER_NI(launch_route, __nv_bfloat16)
                                 : LRM_ROUTER_NI(launch_route, float);
  return go(r, logits, mask, topk_idx, alpha, counts, prob_sum, loss, ws, cs);
}

extern "C" lrm_status lrm_route_bwd(const lrm_router* r, const void* logits, const uint8_t* mask,
                                    const int32_t* topk_idx, const int32_t* counts,
                                    const float* dalpha, const float* dloss, void* dlogits,
                                    void* ws, size_t ws_bytes, void* stream) {
  LRM_NVTX("lrm_route_bwd");
  lrm_status st = check_router(r);
  if (st != LRM_OK) return st;
  if ((st = check_router_ws(r, ws, ws_bytes)) != LRM_OK) return st;
  if (r->T == 0) return LRM_OK;
  if (!logits || !topk_idx || !counts || !dlogits) return LRM_ERR_INVALID_ARG;
  if ((st = check_aligned({logits, topk_idx, counts, dalpha, dloss, dlogits})) != LRM_OK)
    return st;
  cudaStream_t cs = (cudaStream_t)stream;
  auto go = r->dtype == LRM_BF16 ? LRM_ROUTER_NI(launch_route_bwd, __nv_bfloat16)
                                 : LRM_ROUTER_NI(launch_route_bwd, float);
  return go(r, logits, mask, topk_idx, counts, dalpha, dloss, dlogits, error_word(ws), cs);
}
