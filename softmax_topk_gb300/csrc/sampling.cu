// Sampling from rows of logits: the launch.
#include "host_common.h"
#include "internal.h"
#include "kernels/sample_kernel.cuh"

namespace os {

namespace {

template <typename T, int S>
cudaError_t launch_s(const void* x, const float* u, int32_t* out, float* prob, int64_t rows,
                     int cols, const sample::Settings& s, int bits, cudaStream_t stream) {
    return launch_kernel(sample::sample_kernel<T, S>, S * min64(rows, int64_t(1) << 22),
                         sample::kThreads, S, 0, stream, static_cast<const T*>(x), u,
                         reinterpret_cast<int*>(out), prob, rows, cols, s, bits);
}

template <typename T>
cudaError_t launch_t(const void* x, const float* u, int32_t* out, float* prob, int64_t rows,
                     int cols, const sample::Settings& s, cudaStream_t stream) {
    const DeviceInfo* dev = device_info();
    if (!dev) return cudaErrorInvalidDevice;
    // weights are multiples of 2^-bits, at most 1: cols of them fit in 62 bits
    int log2_cols = 0;
    while ((int64_t(1) << log2_cols) < cols) ++log2_cols;
    const int bits = 62 - log2_cols < 44 ? 62 - log2_cols : 44;
    // CTAs per row: as many as the SMs take, while each keeps 32 blocks of 16
    // bytes per warp or more: 8 up to one per SM, 4 up to one and a half, 2 up to
    // two (more of the larger clusters do not all find their place at once).
    // 128256 bf16 columns, us with no filter / top-p 0.9 / top-k 50:
    //   12 rows:  8 13.7/27/21   4 19.1/37/21   2 29.8/58/23   1 46/92/26
    //   38 rows:  8 28.4/57/40   4 27.9/50/23   2 30.1/61/23   1 47/94/27
    //   60 rows:                 4 28.5/52/26   2 30.2/60/24   1 47/93/27
    //   76 rows:                 4 39.6/78/37   2 30.7/60/24   1 47/93/27
    //   152 rows:                               2 53.6/91/34   1 57/106/38
    const int64_t useful = ceil_div(int64_t(cols) * int64_t(sizeof(T)), 16 * sample::kThreads);
    const int64_t half_sms = dev->sms / 2;
    int S = 1;
    if (rows <= 2 * half_sms && useful >= 2) S = 2;
    if (4 * rows <= 3 * half_sms && useful >= 4) S = 4;
    if (8 * rows <= 2 * half_sms && useful >= 8) S = sample::kMaxCluster;
    if (S == 8) return launch_s<T, 8>(x, u, out, prob, rows, cols, s, bits, stream);
    if (S == 4) return launch_s<T, 4>(x, u, out, prob, rows, cols, s, bits, stream);
    if (S == 2) return launch_s<T, 2>(x, u, out, prob, rows, cols, s, bits, stream);
    return launch_s<T, 1>(x, u, out, prob, rows, cols, s, bits, stream);
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
