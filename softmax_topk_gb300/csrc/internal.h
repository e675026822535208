// internal.h -- declarations shared between the C-ABI layer (api.cu) and the
// per-dtype translation units that hold the kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/os_softmax.h"
#include "ctl.h"

namespace os {

#define OS_DECLARE_SOFTMAX_PAIR(NAME)                                                          \
    os_status plan_softmax_##NAME(int64_t rows, int64_t cols, os_path path, bool aligned,      \
                                  os_plan* p);                                                 \
    cudaError_t launch_softmax_##NAME(const os_plan& p, const void* x, void* y, int64_t rows,  \
                                      int cols, bool aligned, int64_t period, int64_t offset,  \
                                      const KernelCtl& ctl, cudaStream_t stream);

OS_DECLARE_SOFTMAX_PAIR(f32_f32)
OS_DECLARE_SOFTMAX_PAIR(bf16_bf16)
OS_DECLARE_SOFTMAX_PAIR(f32_bf16)
OS_DECLARE_SOFTMAX_PAIR(bf16_f32)

os_status plan_topk(int64_t rows, int64_t cols, int K, os_plan* p);
// plain: TopK of x itself (vals = the selected x) instead of softmax + TopK
cudaError_t launch_topk(const os_plan& p, const float* x, float* vals, int32_t* idx,
                        int64_t rows, int cols, int K, bool plain, const KernelCtl& ctl,
                        cudaStream_t stream);

cudaError_t launch_exp(const float* z, float* out, int64_t n, cudaStream_t stream);
// degree 5: the fp32 results' exponential; 3: the bf16 results'
cudaError_t launch_exp_pairs(const float* z, float* out, int64_t n, int degree,
                             cudaStream_t stream);

// one column per row drawn from its K (value, index) pairs, u[r] in [0, 1)
cudaError_t launch_topk_sample(const float* vals, const int32_t* idx, const float* u, int32_t* out,
                               int64_t rows, int K, cudaStream_t stream);

// attention forward over bh slices of [n][d] bf16 (d = 64 or 128): o bf16,
// lse fp32 (may be NULL); scale > 0
cudaError_t launch_attention(const void* q, const void* k, const void* v, void* o, float* lse,
                             int64_t bh, int n, int d, float scale, bool causal,
                             const KernelCtl& ctl, cudaStream_t stream);

// gradient of the attention forward; delta is a workspace of bh * n floats,
// dlse (the gradient that reaches the logsumexp) may be NULL
struct AttentionBwdArgs {
    const void *q, *k, *v, *o, *dout;
    const float *lse, *dlse;
    void *dq, *dk, *dv;
    float* delta;
    int64_t bh;
    int n;
    float scale;
    bool causal;
};
cudaError_t launch_attention_bwd(const AttentionBwdArgs& a, int d, const KernelCtl& ctl,
                                 cudaStream_t stream);

// router over experts (see os_route_topk, os_route_bwd)
struct RouteArgs {
    const void* x;
    os_dtype in;
    const float* bias;  // or NULL
    int64_t rows;
    int experts, K, groups, topk_groups, group_top;
    os_score score;
    bool renorm;
    float scale;
};
#define OS_DECLARE_ROUTE(NAME)                                                                \
    cudaError_t route_fwd_##NAME(const RouteArgs& a, float* weights, int32_t* idx,            \
                                 cudaStream_t stream);                                        \
    cudaError_t route_bwd_##NAME(const RouteArgs& a, const int32_t* idx,                      \
                                 const float* dweights, void* dx, cudaStream_t stream);

OS_DECLARE_ROUTE(f32)
OS_DECLARE_ROUTE(bf16)

// one column per row under the sampling settings (see os_sample)
cudaError_t launch_sample(const void* x, os_dtype in, const float* u, int32_t* out, float* prob,
                          int64_t rows, int cols, const os_sampling& s, cudaStream_t stream);

// paged key-value cache (see os_paged_append, os_paged_attention, os_paged_reorder)
struct PagedAppendArgs {
    const void *q, *k, *v;  // q may be NULL
    int64_t q_stride, k_stride, v_stride;
    void* q_out;
    const int32_t* starts;  // or NULL
    const float* inv_freq;  // or NULL
    int64_t tokens;
    int q_heads, rot;
    bool interleaved;
};
cudaError_t launch_paged_append(const os_paged_cache& c, const PagedAppendArgs& p,
                                cudaStream_t stream);
cudaError_t launch_paged_reorder(const os_paged_cache& c, const int32_t* parents, int beams,
                                 int layers, int32_t* out_table, int32_t* out_lengths,
                                 cudaStream_t stream);
constexpr float kScoreLog2e = 1.44269504f;
int64_t paged_attention_workspace(int sms);
cudaError_t launch_paged_attention(const os_paged_cache& c, const void* q, int64_t q_stride,
                                   void* out, float* lse, void* workspace, int q_heads, float scale,
                                   cudaStream_t stream);

// beam search's selection (see os_beam_select)
struct BeamSelectArgs {
    const void* x;
    os_dtype in;
    const float* scores;
    const uint8_t* ended;  // or NULL
    float* out;
    int32_t *parents, *tokens;
    void* workspace;
    int64_t groups, cols;
    int beams, K, pad;
};
int64_t beam_select_workspace(int64_t groups, int beams, int64_t cols, int K, os_dtype in, int sms);
cudaError_t launch_beam_select(const BeamSelectArgs& p, cudaStream_t stream);

// (m, d, lse) of every row; any output may be NULL
cudaError_t launch_stats(const void* x, os_dtype in, float* m, float* d, float* lse, int64_t rows,
                         int cols, bool aligned, cudaStream_t stream);

}  // namespace os
