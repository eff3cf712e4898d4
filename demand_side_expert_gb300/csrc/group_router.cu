// Entry points of the grouped router (the kernels: group_router.cuh), and its bias's step.
#include "group_router.h"
#include "router.cuh"

namespace lrm {

constexpr int kMaxGroups = 32;

__global__ void bias_step_kernel(const int32_t* __restrict__ counts, const float* bias, float* out,
                                 int E, float rate) {
  pdl_begin();  // predecessor complete before any global access
  __shared__ long long red[32];
  long long sum = 0;
  for (int e = threadIdx.x; e < E; e += blockDim.x) sum += counts[e];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) sum += red[w];
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    const long long lack = sum - (long long)E * counts[e];
    out[e] = bias[e] + (lack > 0 ? rate : lack < 0 ? -rate : 0.f);
  }
}

static lrm_status check_group_router(const lrm_group_router* r) {
  if (!r) return LRM_ERR_INVALID_ARG;
  if (r->T < 0 || r->E <= 0 || r->K <= 0 || r->groups <= 0 || r->top_groups <= 0 ||
      r->group_top <= 0)
    return LRM_ERR_INVALID_ARG;
  if (r->dtype != LRM_F32 && r->dtype != LRM_BF16) return LRM_ERR_INVALID_ARG;
  if (r->score_fn != LRM_SIGMOID && r->score_fn != LRM_SOFTMAX) return LRM_ERR_INVALID_ARG;
  if (r->stride < r->E) return LRM_ERR_INVALID_ARG;
  if (r->E > kRouterMaxE || r->K > kRouterMaxK || r->groups > kMaxGroups || r->group_top > 2)
    return LRM_ERR_UNSUPPORTED;
  if (r->E % r->groups != 0 || r->top_groups > r->groups ||
      r->K > r->top_groups * (r->E / r->groups))
    return LRM_ERR_UNSUPPORTED;
  if ((int64_t)r->T * r->K >= (int64_t)1 << 31) return LRM_ERR_UNSUPPORTED;
  return LRM_OK;
}

static size_t group_router_bytes(const lrm_group_router* r) {
  // header, then sums of the shares and counts of every CTA
  return kWsHeaderBytes + ((size_t)kRouterMaxCtas * 8 * r->E + 255) / 256 * 256;
}

static lrm_status check_group_ws(const lrm_group_router* r, const void* ws, size_t ws_bytes) {
  if (!ws) return LRM_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return LRM_ERR_UNSUPPORTED;
  return ws_bytes < group_router_bytes(r) ? LRM_ERR_WORKSPACE : LRM_OK;
}

}  // namespace lrm

using namespace lrm;

extern "C" size_t lrm_group_router_workspace_bytes(const lrm_group_router* r) {
  return check_group_router(r) == LRM_OK ? group_router_bytes(r) : 0;
}

extern "C" lrm_status lrm_group_route(const lrm_group_router* r, const void* logits,
                                      const float* bias, const uint8_t* mask, int32_t* topk_idx,
                                      float* alpha, int32_t* counts, float* prob_sum, float* loss,
                                      void* ws, size_t ws_bytes, void* stream) {
  LRM_NVTX("lrm_group_route");
  lrm_status st = check_group_router(r);
  if (st != LRM_OK) return st;
  if ((st = check_group_ws(r, ws, ws_bytes)) != LRM_OK) return st;
  const int given = !!counts + !!prob_sum + !!loss;
  if (given != 0 && given != 3) return LRM_ERR_INVALID_ARG;
  if (r->T > 0 && (!logits || !topk_idx || !alpha)) return LRM_ERR_INVALID_ARG;
  if ((st = check_aligned({logits, topk_idx, alpha, counts, prob_sum})) != LRM_OK) return st;
  if (((reinterpret_cast<uintptr_t>(bias) | reinterpret_cast<uintptr_t>(loss)) & 3) != 0)
    return LRM_ERR_UNSUPPORTED;
  if (r->T == 0 && !counts) return LRM_OK;
  // all groups kept are one group of all experts
  const int groups = r->top_groups == r->groups ? 1 : r->groups;
  RouteArgs a{bias, mask, topk_idx, alpha, counts, prob_sum, loss,
              reinterpret_cast<float2*>((char*)ws + kWsHeaderBytes), r->stride, r->T, r->E, r->K,
              0, r->score_fn == LRM_SOFTMAX, groups, r->E / groups, r->top_groups,
              r->group_top, r->renorm, r->scale, r->balance_coef};
  cudaStream_t cs = (cudaStream_t)stream;
  return r->dtype == LRM_BF16 ? group_route_bf16(logits, a, cs)
                              : group_route_f32(logits, a, cs);
}

extern "C" lrm_status lrm_group_route_bwd(const lrm_group_router* r, const void* logits,
                                          const uint8_t* mask, const int32_t* topk_idx,
                                          const int32_t* counts, const float* dalpha,
                                          const float* dloss, void* dlogits, void* ws,
                                          size_t ws_bytes, void* stream) {
  LRM_NVTX("lrm_group_route_bwd");
  lrm_status st = check_group_router(r);
  if (st != LRM_OK) return st;
  if ((st = check_group_ws(r, ws, ws_bytes)) != LRM_OK) return st;
  if (r->T == 0) return LRM_OK;
  if (!logits || !topk_idx || !counts || !dlogits) return LRM_ERR_INVALID_ARG;
  if ((st = check_aligned({logits, topk_idx, counts, dalpha, dlogits})) != LRM_OK) return st;
  if ((reinterpret_cast<uintptr_t>(dloss) & 3) != 0) return LRM_ERR_UNSUPPORTED;
  const RouteBwdArgs a{mask, topk_idx, counts, dalpha, dloss, r->stride, r->T, r->E, r->K, 0, 0,
                       r->score_fn == LRM_SOFTMAX, r->renorm, r->scale, r->balance_coef,
                       error_word(ws)};
  cudaStream_t cs = (cudaStream_t)stream;
  return r->dtype == LRM_BF16 ? group_route_bwd_bf16(logits, a, dlogits, cs)
                              : group_route_bwd_f32(logits, a, dlogits, cs);
}

extern "C" lrm_status lrm_bias_step(const lrm_bias* b, const int32_t* counts, const float* bias,
                                    float* out, void* stream) {
  LRM_NVTX("lrm_bias_step");
  if (!b || !counts || !bias || !out || b->E <= 0) return LRM_ERR_INVALID_ARG;
  if (b->E > kRouterMaxE) return LRM_ERR_UNSUPPORTED;
  if (((reinterpret_cast<uintptr_t>(counts) | reinterpret_cast<uintptr_t>(bias) |
        reinterpret_cast<uintptr_t>(out)) & 3) != 0)
    return LRM_ERR_UNSUPPORTED;
  launch_k(bias_step_kernel, dim3(1), dim3((b->E + 31) / 32 * 32), 0, (cudaStream_t)stream, counts,
           bias, out, b->E, b->rate);
  return launch_status();
}
