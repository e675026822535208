// Router over experts, f32 logits.
#include "route_dispatch.cuh"

namespace os {

cudaError_t route_fwd_f32(const RouteArgs& a, float* weights, int32_t* idx, cudaStream_t stream) {
    return fwd<float>(a, weights, idx, stream);
}
cudaError_t route_bwd_f32(const RouteArgs& a, const int32_t* idx, const float* dweights, void* dx,
                         cudaStream_t stream) {
    return bwd<float>(a, idx, dweights, dx, stream);
}

}  // namespace os
