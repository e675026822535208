// Attention gradient: the row constants delta, then the two tensor-core
// kernels (dK and dV by key tiles, dQ by query tiles).
#include <cuda.h>

#include "host_common.h"
#include "internal.h"
#include "kernels/attention_bwd_kernel.cuh"
#include "tensor_map.h"

namespace os {

namespace {

using attn_bwd::Side;

template <int D>
cudaError_t launch_d(const AttentionBwdArgs& a, const KernelCtl& ctl, cudaStream_t stream) {
    const DeviceInfo* dev = device_info();
    if (!dev) return cudaErrorInvalidDevice;
    Side kv = {}, q = {};
    if (!make_tile_map(&kv.x, a.k, a.bh, a.n, D) || !make_tile_map(&kv.y, a.v, a.bh, a.n, D) ||
        !make_tile_map(&kv.u, a.q, a.bh, a.n, D) || !make_tile_map(&kv.w, a.dout, a.bh, a.n, D))
        return cudaErrorInvalidValue;
    kv.out1 = static_cast<__nv_bfloat16*>(a.dk);
    kv.out2 = static_cast<__nv_bfloat16*>(a.dv);
    q.x = kv.u;
    q.y = kv.w;
    q.u = kv.x;
    q.w = kv.y;
    q.out1 = static_cast<__nv_bfloat16*>(a.dq);
    const int64_t rows = a.bh * a.n;
    cudaError_t e = launch_kernel(attn_bwd::delta_kernel<D>, ceil_div(rows * (D / 8), 256), 256, 1,
                                  0, stream, static_cast<const __nv_bfloat16*>(a.o),
                                  static_cast<const __nv_bfloat16*>(a.dout), a.dlse, a.delta, rows);
    if (e != cudaSuccess) return e;
    const int nt = static_cast<int>(ceil_div(a.n, attn_bwd::kRows));
    const int64_t units = a.causal ? a.bh * ((nt + 1) / 2) : a.bh * nt;
    // both sides in one launch, each by as many CTAs as it has units or the GPU
    // SMs; those of the second side start as the first side's leave
    const int ctas = static_cast<int>(min64(units, dev->sms));
    auto k = attn_bwd::attention_bwd_kernel<D>;
    constexpr int smem = attn_bwd::Layout<D>::kBytes;
    if (!prepare_kernel(k, 1, smem)) return cudaErrorInvalidConfiguration;
    return launch_kernel(k, 2 * ctas, attn_bwd::kThreads, 1, smem, stream, kv, q, a.lse,
                         static_cast<const float*>(a.delta), a.n, nt, static_cast<int>(units),
                         a.scale, a.causal ? 1 : 0, ctl);
}

}  // namespace

cudaError_t launch_attention_bwd(const AttentionBwdArgs& a, int d, const KernelCtl& ctl,
                                 cudaStream_t stream) {
    return d == 64 ? launch_d<64>(a, ctl, stream) : launch_d<128>(a, ctl, stream);
}

}  // namespace os
