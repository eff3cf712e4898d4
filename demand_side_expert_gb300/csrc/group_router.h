// Arguments of the grouped router's kernels, and their launchers by the logits' type.
#pragma once

#include "common.cuh"

namespace lrm {

struct RouteArgs {
  const float* bias;
  const uint8_t* mask;
  int32_t* topk_idx;
  float* alpha;
  int32_t* counts;
  float *prob_sum, *loss;
  float2* part;
  int64_t stride;
  int ntok, E, K, vec, softmax, groups, size, top_groups, group_top, renorm;
  float scale, balance_coef;
};

struct RouteBwdArgs {
  const uint8_t* mask;
  const int32_t *topk_idx, *counts;
  const float *dalpha, *dloss;
  int64_t stride;
  int ntok, E, K, vec, out_vec, softmax, renorm;
  float scale, balance_coef;
  int32_t* err;
};

// One translation unit a type: their many instantiations compile side by side.
lrm_status group_route_bf16(const void* logits, const RouteArgs& a, cudaStream_t cs);
lrm_status group_route_f32(const void* logits, const RouteArgs& a, cudaStream_t cs);
lrm_status group_route_bwd_bf16(const void* logits, const RouteBwdArgs& a, void* dlogits,
                                cudaStream_t cs);
lrm_status group_route_bwd_f32(const void* logits, const RouteBwdArgs& a, void* dlogits,
                               cudaStream_t cs);

}  // namespace lrm
