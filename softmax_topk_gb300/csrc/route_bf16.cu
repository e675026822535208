// Router over experts, bf16 logits.
#include "route_dispatch.cuh"

namespace os {

cudaError_t route_fwd_bf16(const RouteArgs& a, float* weights, int32_t* idx, cudaStream_t stream) {
    return fwd<__nv_bfloat16>(a, weights, idx, stream);
}
cudaError_t route_bwd_bf16(const RouteArgs& a, const int32_t* idx, const float* dweights, void* dx,
                         cudaStream_t stream) {
    return bwd<__nv_bfloat16>(a, idx, dweights, dx, stream);
}

}  // namespace os
