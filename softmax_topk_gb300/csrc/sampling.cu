// Sampling from rows of logits: the launch.
#include "host_common.h"
#include "internal.h"
#include "kernels/sample_kernel.cuh"

namespace os {

namespace {

template <typename T>
cudaError_t launch_t(const void* x, const float* u, int32_t* out, float* prob, int64_t rows,
                     int cols, const sample::Settings& s, cudaStream_t stream) {
    // weights are multiples of 2^-bits, at most 1: cols of them fit in 62 bits
    int log2_cols = 0;
    while ((int64_t(1) << log2_cols) < cols) ++log2_cols;
    const int bits = 62 - log2_cols < 44 ? 62 - log2_cols : 44;
    return launch_kernel(sample::sample_kernel<T>, min64(rows, int64_t(1) << 22),
                         sample::kThreads, 1, 0, stream, static_cast<const T*>(x), u,
                         reinterpret_cast<int*>(out), prob, rows, cols, s, bits);
}

}  // namespace

cudaError_t launch_sample(const void* x, os_dtype in, const float* u, int32_t* out, float* prob,
                          int64_t rows, int cols, const os_sampling& p, cudaStream_t stream) {
    sample::Settings s = {};
    s.temperature = p.temperature;
    s.top_k = reinterpret_cast<const int*>(p.top_k);
    s.top_p = p.top_p;
    s.min_p = p.min_p;
    s.temperature_all = p.temperature_all;
    s.top_k_all = p.top_k_all;
    s.top_p_all = p.top_p_all;
    s.min_p_all = p.min_p_all;
    return in == OS_F32 ? launch_t<float>(x, u, out, prob, rows, cols, s, stream)
                        : launch_t<__nv_bfloat16>(x, u, out, prob, rows, cols, s, stream);
}

}  // namespace os
