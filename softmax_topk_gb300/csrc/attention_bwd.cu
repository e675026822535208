// Attention gradient: the row constants delta, then the two tensor-core
// kernels (dK and dV by key tiles, dQ by query tiles).
#include <cuda.h>

#include "host_common.h"
#include "internal.h"
#include "kernels/attention_bwd_kernel.cuh"
#include "tensor_map.h"

namespace os {

namespace {

template <int D, bool KV>
cudaError_t launch_side(const CUtensorMap& mx, const CUtensorMap& my, const CUtensorMap& mu,
                        const CUtensorMap& mw, const float* lse, const float* delta, void* out1,
                        void* out2, int64_t bh, int n, float scale, bool causal,
                        const KernelCtl& ctl, cudaStream_t stream) {
    auto k = attn_bwd::attention_bwd_kernel<D, KV>;
    constexpr int smem = attn_bwd::Layout<D>::kBytes;
    if (!prepare_kernel(k, 1, smem)) return cudaErrorInvalidConfiguration;
    const DeviceInfo* dev = device_info();
    if (!dev) return cudaErrorInvalidDevice;
    const int nt = (n + attn_bwd::kRows - 1) / attn_bwd::kRows;
    const int64_t units = causal ? bh * ((nt + 1) / 2) : bh * nt;
    return launch_kernel(k, min64(units, dev->sms), attn_bwd::kThreads, 1, smem, stream, mx, my, mu,
                         mw, lse, delta, static_cast<__nv_bfloat16*>(out1),
                         static_cast<__nv_bfloat16*>(out2), n, nt, static_cast<int>(units), scale,
                         causal ? 1 : 0, ctl);
}

template <int D>
cudaError_t launch_d(const AttentionBwdArgs& a, const KernelCtl& ctl, cudaStream_t stream) {
    CUtensorMap mq, mk, mv, mdo;
    if (!make_tile_map(&mq, a.q, a.bh, a.n, D) || !make_tile_map(&mk, a.k, a.bh, a.n, D) ||
        !make_tile_map(&mv, a.v, a.bh, a.n, D) || !make_tile_map(&mdo, a.dout, a.bh, a.n, D))
        return cudaErrorInvalidValue;
    const int64_t rows = a.bh * a.n;
    cudaError_t e = launch_kernel(attn_bwd::delta_kernel<D>, ceil_div(rows * (D / 8), 256), 256, 1,
                                  0, stream, static_cast<const __nv_bfloat16*>(a.o),
                                  static_cast<const __nv_bfloat16*>(a.dout), a.dlse, a.delta, rows);
    if (e != cudaSuccess) return e;
    e = launch_side<D, true>(mk, mv, mq, mdo, a.lse, a.delta, a.dk, a.dv, a.bh, a.n, a.scale,
                             a.causal, ctl, stream);
    if (e != cudaSuccess) return e;
    return launch_side<D, false>(mq, mdo, mk, mv, a.lse, a.delta, a.dq, nullptr, a.bh, a.n, a.scale,
                                 a.causal, ctl, stream);
}

}  // namespace

cudaError_t launch_attention_bwd(const AttentionBwdArgs& a, int d, const KernelCtl& ctl,
                                 cudaStream_t stream) {
    return d == 64 ? launch_d<64>(a, ctl, stream) : launch_d<128>(a, ctl, stream);
}

}  // namespace os
