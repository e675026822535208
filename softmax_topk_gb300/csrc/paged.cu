// Paged key-value cache: the append with rotation, and the reordering of states
// that follows a beam search's choice.
#include "host_common.h"
#include "internal.h"
#include "kernels/paged_kernels.cuh"

namespace os {

namespace {

template <int D, bool INTERLEAVED>
cudaError_t append(const paged::AppendArgs& a, cudaStream_t stream) {
    // One token per CTA until the GPU is full of them, then four: angles and places
    // are worked out for all at once.  us with one / four: 512 tokens 3.6 / 4.1, 1000
    // 5.3 / 5.6, 2400 8.7 / 7.7, 5000 16.3 / 13.0, 36000 92 / 69 (16 + 8 heads of 128).
    const DeviceInfo* dev = device_info();
    if (!dev) return cudaErrorInvalidDevice;
    const int per_cta = a.tokens >= 16 * int64_t(dev->sms) ? paged::kAppendTokens : 1;
    return launch_behind(paged::append_kernel<D, INTERLEAVED>,
                         dim3(static_cast<unsigned>(ceil_div(a.tokens, per_cta))),
                         paged::kAppendThreads, 0, stream, a, per_cta);
}

}  // namespace

cudaError_t launch_paged_append(const os_paged_cache& c, const PagedAppendArgs& p,
                                cudaStream_t stream) {
    paged::AppendArgs a = {};
    a.k_cache = static_cast<__nv_bfloat16*>(c.k);
    a.v_cache = static_cast<__nv_bfloat16*>(c.v);
    a.table = c.table;
    a.lengths = c.lengths;
    a.q = static_cast<const __nv_bfloat16*>(p.q);
    a.k = static_cast<const __nv_bfloat16*>(p.k);
    a.v = static_cast<const __nv_bfloat16*>(p.v);
    a.q_out = static_cast<__nv_bfloat16*>(p.q_out);
    a.starts = p.starts;
    a.inv_freq = p.inv_freq;
    a.q_stride = p.q_stride;
    a.k_stride = p.k_stride;
    a.v_stride = p.v_stride;
    a.tokens = p.tokens;
    a.seqs = static_cast<int>(c.seqs);
    a.width = static_cast<int>(c.width);
    a.pages = static_cast<int>(c.pages);
    a.kv_heads = c.kv_heads;
    a.q_heads = p.q ? p.q_heads : 0;
    a.rot = p.inv_freq ? p.rot : 0;
    a.split = paged::page_split(c.page_size);
    if (c.head_dim == 64)
        return p.interleaved ? append<64, true>(a, stream) : append<64, false>(a, stream);
    return p.interleaved ? append<128, true>(a, stream) : append<128, false>(a, stream);
}

cudaError_t launch_paged_reorder(const os_paged_cache& c, const int32_t* parents, int beams,
                                 int layers, int32_t* out_table, int32_t* out_lengths,
                                 cudaStream_t stream) {
    paged::ReorderArgs a = {};
    a.k_cache = static_cast<__nv_bfloat16*>(c.k);
    a.v_cache = static_cast<__nv_bfloat16*>(c.v);
    a.table = c.table;
    a.lengths = c.lengths;
    a.parents = parents;
    a.out_table = out_table;
    a.out_lengths = out_lengths;
    a.row_bytes = c.head_dim * 2;
    a.head_bytes = a.row_bytes * c.page_size;
    a.page_bytes = a.head_bytes * c.kv_heads;
    a.layer_bytes = a.page_bytes * c.pages;
    a.seqs = static_cast<int>(c.seqs);
    a.beams = beams;
    a.width = static_cast<int>(c.width);
    a.pages = static_cast<int>(c.pages);
    a.kv_heads = c.kv_heads;
    a.layers = layers;
    a.split = paged::page_split(c.page_size);
    return launch_behind(paged::reorder_kernel,
                         dim3(static_cast<unsigned>(c.seqs * layers * c.kv_heads)),
                         paged::kReorderThreads, 0, stream, a);
}

}  // namespace os
