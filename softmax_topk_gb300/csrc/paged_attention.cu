// Attention of one new token per sequence over a paged key-value cache: the split
// kernel and, where units span CTAs, the join.
#include "host_common.h"
#include "internal.h"
#include "kernels/paged_attention_kernel.cuh"

namespace os {

namespace {

// Blocks that a CTA should have at least: fewer CTAs leave fewer pieces to join.  us with
// 2, 4, 8, 16 blocks, 2 key heads: 300 keys 6.5 / 6.2 / 7.0 / 7.6, 1000 keys 7.2 / 6.8 /
// 7.4 / 8.3, 3000 keys 9.4 / 8.2 / 7.9 / 8.5.
constexpr int kMinBlocks = 4;

template <int D, int NT>
int64_t workspace_bytes(int ctas) {
    using S = paged::AttnShape<D, NT>;
    return ctas * int64_t(sizeof(int4) + 2 * S::kPiece * sizeof(float));
}

template <int D, int NT>
cudaError_t launch(paged::AttnArgs a, void* workspace, cudaStream_t stream) {
    using S = paged::AttnShape<D, NT>;
    const DeviceInfo* dev = device_info();
    if (!dev) return cudaErrorInvalidDevice;
    a.chunks = static_cast<int>(ceil_div(a.group, S::kHeads));
    a.units = a.kv_heads * a.chunks;
    const int64_t most =
        ceil_div(int64_t(a.width) * a.split.size, paged::kBlock) * a.seqs * a.units;
    const int ctas = static_cast<int>(min64(dev->sms, ceil_div(most, kMinBlocks)));
    a.ctas = ctas;
    a.tails = static_cast<int4*>(workspace);
    a.parts = reinterpret_cast<float*>(a.tails + ctas);
    auto k = paged::paged_attention_kernel<D, NT>;
    constexpr int smem = sizeof(paged::AttnShared<D, NT>);
    if (!prepare_kernel(k, 1, smem)) return cudaErrorInvalidConfiguration;
    const cudaError_t e = launch_behind(k, dim3(ctas), S::kThreads, smem, stream, a);
    if (e != cudaSuccess || ctas == 1) return e;
    const unsigned heads = static_cast<unsigned>(min64(a.group, S::kHeads));
    const bool by_unit = int64_t(a.seqs) * a.units < ctas;
    return launch_behind(by_unit ? paged::paged_join_kernel<D, NT, true>
                                 : paged::paged_join_kernel<D, NT, false>,
                         dim3(by_unit ? static_cast<unsigned>(a.seqs * a.units) : ctas, heads),
                         32 * paged::join_warps(by_unit), 0, stream, a);
}

}  // namespace

int64_t paged_attention_workspace(int sms) { return workspace_bytes<128, 2>(sms); }

cudaError_t launch_paged_attention(const os_paged_cache& c, const void* q, int64_t q_stride,
                                   void* out, float* lse, void* workspace, int q_heads, float scale,
                                   cudaStream_t stream) {
    paged::AttnArgs a = {};
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k = static_cast<const __nv_bfloat16*>(c.k);
    a.v = static_cast<const __nv_bfloat16*>(c.v);
    a.table = c.table;
    a.lengths = c.lengths;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.q_stride = q_stride;
    a.seqs = static_cast<int>(c.seqs);
    a.width = static_cast<int>(c.width);
    a.pages = static_cast<int>(c.pages);
    a.kv_heads = c.kv_heads;
    a.group = q_heads / c.kv_heads;
    a.scale_log2 = scale * 1.44269504f;
    a.split = paged::page_split(c.page_size);
    if (c.head_dim == 64)
        return a.group <= 8 ? launch<64, 1>(a, workspace, stream) : launch<64, 2>(a, workspace, stream);
    return a.group <= 8 ? launch<128, 1>(a, workspace, stream) : launch<128, 2>(a, workspace, stream);
}

}  // namespace os
