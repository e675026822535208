// Attention of one new token per sequence over a paged key-value cache: the split
// kernel and, where units span CTAs, the join.
#include "host_common.h"
#include "internal.h"
#include "kernels/paged_attention_kernel.cuh"

namespace os {

namespace {

// Blocks of the table's room per CTA, at least: fewer CTAs leave fewer pieces to join.  us
// with 2, 4, 8 blocks, 2 key heads and tables no wider than the sequence: 300 keys 6.1 / 6.1 /
// 6.9, 1000 keys 6.7 / 6.4 / 6.9, 3000 keys 6.9 / 7.1 / 7.2.  The host knows the room alone.
// Under a wide table there is a CTA per SM, whatever the lengths, down to a block each.  us
// for a table of 131072 keys, in brackets for one that fits: 1 x 300, 2 x 8 heads 6.0 (6.1),
// 1 x 1000 6.5 (6.5), 1 x 2000, 16 heads on one 8.7 (7.4), 4 x 200, 16 on one 6.7 (7.7),
// 64 x 40, 2 x 4 heads 6.9 (7.0), 100 x 33, 8 heads of 64 on one 10.3 (7.1).  Four blocks at
// least by the lengths, in both kernels, took 6.1, 6.5, 7.6, 7.6, 8.9 and 11.1 there.
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
    // Sixteen warps a head where the join has an SM for each, else four.  us with sixteen,
    // eight, four: 1 x 1000, 2 x 8 heads 6.5 / 6.8 / 6.7, 1 x 131072 28.6 / 30.0 / 32.4,
    // 2 x 30000, 2 x 16 heads 18.4 / 19.1 / 20.4; 64 x 4096, 16 heads on one 43.5 / 35.9 /
    // 31.9, 16 x 4096, 4 x 8 heads 32.2 / 28.8 / 27.7.
    const int64_t units = int64_t(a.seqs) * a.units, heads = min64(a.group, S::kHeads);
    const bool by_unit = units < ctas;
    const bool many = by_unit && units * heads <= dev->sms;
    constexpr int kMany = paged::kJoinWarps, kFew = paged::kFewJoinWarps;
    return launch_behind(many      ? paged::paged_join_kernel<D, NT, true, kMany>
                         : by_unit ? paged::paged_join_kernel<D, NT, true, kFew>
                                   : paged::paged_join_kernel<D, NT, false, kFew>,
                         dim3(static_cast<unsigned>(by_unit ? units : ctas),
                              static_cast<unsigned>(heads)),
                         32 * (many ? kMany : kFew), 0, stream, a);
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
    a.scale_log2 = scale * kScoreLog2e;
    a.split = paged::page_split(c.page_size);
    if (c.head_dim == 64)
        return a.group <= 8 ? launch<64, 1>(a, workspace, stream) : launch<64, 2>(a, workspace, stream);
    return a.group <= 8 ? launch<128, 1>(a, workspace, stream) : launch<128, 2>(a, workspace, stream);
}

}  // namespace os
