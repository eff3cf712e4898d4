#include "group_router.cuh"

namespace lrm {

lrm_status group_route_bf16(const void* logits, const RouteArgs& a, cudaStream_t cs) {
  return pick_group_route<__nv_bfloat16>(logits, a, cs);
}

lrm_status group_route_bwd_bf16(const void* logits, const RouteBwdArgs& a, void* dlogits,
                              cudaStream_t cs) {
  return pick_group_bwd<__nv_bfloat16>(logits, a, dlogits, cs);
}

}  // namespace lrm
