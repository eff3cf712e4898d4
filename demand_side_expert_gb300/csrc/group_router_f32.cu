#include "group_router.cuh"

namespace lrm {

lrm_status group_route_f32(const void* logits, const RouteArgs& a, cudaStream_t cs) {
  return pick_group_route<float>(logits, a, cs);
}

lrm_status group_route_bwd_f32(const void* logits, const RouteBwdArgs& a, void* dlogits,
                              cudaStream_t cs) {
  return pick_group_bwd<float>(logits, a, dlogits, cs);
}

}  // namespace lrm
