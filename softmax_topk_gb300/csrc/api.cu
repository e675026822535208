// api.cu -- the C ABI declared in include/os_softmax.h: argument checks, kernel
// choice per dtype pair, launch on the caller's stream.  No allocation, no
// synchronisation, no host fallback.
#include <atomic>
#include <cstdint>

#include "host_common.h"
#include "internal.h"

// Device status word (one per device the library runs on): kernels OR in
// os::kErrWaitTimeout when a bounded wait gives up.  Read and cleared in one
// atomic exchange by os_device_status, whose result lands in the second word.
__device__ unsigned int os_device_status_word;
__device__ unsigned int os_device_status_taken;

// The status word's value at the moment it is cleared: a timeout recorded by a
// kernel on another stream lands either before the exchange (and is reported
// now) or after it (and is reported by the next call), never lost between a
// read and a separate clear.
__global__ void status_exchange_kernel() {
    os_device_status_taken = atomicExch(&os_device_status_word, 0u);
}

namespace {

std::atomic<unsigned long long> g_timeout_ns{1000000000ull};  // 1 s per wait
std::atomic<int> g_fault{0};

// Address of this device's status word (host code cannot use the symbol
// itself as a device pointer), looked up once per device.
unsigned int* status_word() {
    constexpr int kMaxDevices = 64;
    static unsigned int* cache[kMaxDevices] = {nullptr};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!cache[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, os_device_status_word) != cudaSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        cache[dev] = static_cast<unsigned int*>(p);
    }
    return cache[dev];
}

bool make_ctl(os::KernelCtl* ctl) {
    ctl->err = status_word();
    ctl->timeout_ns = g_timeout_ns.load();
    ctl->fault = g_fault.load();
    return ctl->err != nullptr;
}

using PlanFn = os_status (*)(int64_t, int64_t, os_path, bool, os_plan*);
using LaunchFn = cudaError_t (*)(const os_plan&, const void*, void*, int64_t, int, bool, int64_t,
                                 int64_t, const os::KernelCtl&, cudaStream_t);

struct Pair {
    PlanFn plan;
    LaunchFn launch;
};

// [in_dtype][out_dtype]
const Pair kPairs[2][2] = {
    {{os::plan_softmax_f32_f32, os::launch_softmax_f32_f32},
     {os::plan_softmax_f32_bf16, os::launch_softmax_f32_bf16}},
    {{os::plan_softmax_bf16_f32, os::launch_softmax_bf16_f32},
     {os::plan_softmax_bf16_bf16, os::launch_softmax_bf16_bf16}},
};

bool valid_dtype(int t) { return t == OS_F32 || t == OS_BF16; }
int64_t elem_bytes(os_dtype t) { return t == OS_F32 ? 4 : 2; }
int elems_per_vector(os_dtype t) { return t == OS_F32 ? 4 : 8; }

bool overlaps(const void* a, int64_t na, const void* b, int64_t nb) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return pa < pb + uintptr_t(nb) && pb < pa + uintptr_t(na);
}

// A buffer of a call; those that are NULL are passed over.
struct Buffer {
    const void* p;
    int64_t bytes;
};

// No written buffer overlaps a read one or another written one.
template <int W, int R>
bool apart(const Buffer (&written)[W], const Buffer (&read)[R]) {
    for (int i = 0; i < W; ++i) {
        if (!written[i].p) continue;
        for (const Buffer& r : read)
            if (r.p && overlaps(written[i].p, written[i].bytes, r.p, r.bytes)) return false;
        for (int j = 0; j < i; ++j)
            if (written[j].p &&
                overlaps(written[i].p, written[i].bytes, written[j].p, written[j].bytes))
                return false;
    }
    return true;
}

// rows >= 0, 1 <= cols <= 2^31-1, and rows*cols*8 representable.
bool shape_ok(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 1 || cols > INT32_MAX) return false;
    return rows <= INT64_MAX / 8 / cols;
}

os_status softmax_checks(int64_t rows, int64_t cols, os_dtype in, os_dtype out, os_path path) {
    if (!valid_dtype(in) || !valid_dtype(out)) return OS_ERR_DTYPE;
    if (!shape_ok(rows, cols)) return OS_ERR_SHAPE;
    if (path < OS_PATH_AUTO || path > OS_PATH_STREAM_POLY) return OS_ERR_PATH;
    return OS_OK;
}

os_status topk_checks(int64_t rows, int64_t cols, int32_t K) {
    if (!shape_ok(rows, cols)) return OS_ERR_SHAPE;
    if (K < 1 || K > 256 || int64_t(K) > cols) return OS_ERR_K;
    return OS_OK;
}

// period > 0: causal mask; only the WARP and STREAM families take one, and AUTO
// picks between those two.
os_status softmax_entry(const void* x, void* y, int64_t rows, int64_t cols, os_dtype in,
                        os_dtype out, os_path path, int64_t period, int64_t offset,
                        os_stream_t stream) {
    os_status st = softmax_checks(rows, cols, in, out, path);
    if (st != OS_OK) return st;
    if (rows == 0) return OS_OK;
    if (!x || !y) return OS_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(x) % elem_bytes(in) ||
        reinterpret_cast<uintptr_t>(y) % elem_bytes(out))
        return OS_ERR_ALIGN;
    // exactly in place (y == x, one dtype) is allowed: every kernel family
    // reads each element of a row before the same thread or CTA writes it;
    // any other overlap is not
    const bool in_place = x == y && in == out;
    if (!in_place && overlaps(x, rows * cols * elem_bytes(in), y, rows * cols * elem_bytes(out)))
        return OS_ERR_ALIAS;
    const bool ptrs_aligned = reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                              reinterpret_cast<uintptr_t>(y) % 16 == 0;
    if (period > 0) {
        // the vector slots a row needs (one more when rows are not 16-byte
        // aligned whole vectors), as the plan counts them
        const int epv = elems_per_vector(in);
        const int64_t nv = (ptrs_aligned && cols % epv == 0) ? (cols + epv - 1) / epv
                                                             : (cols + 2 * epv - 2) / epv;
        if (path == OS_PATH_AUTO) path = nv <= 256 ? OS_PATH_WARP : OS_PATH_STREAM;
        if (path != OS_PATH_WARP && path != OS_PATH_STREAM && path != OS_PATH_STREAM_POLY)
            return OS_ERR_PATH;
    }
    os_plan plan;
    st = kPairs[in][out].plan(rows, cols, path, ptrs_aligned, &plan);
    if (st != OS_OK) return st;
    os::KernelCtl ctl;
    if (!make_ctl(&ctl)) return OS_ERR_CUDA;
    const bool aligned = ptrs_aligned && cols % elems_per_vector(in) == 0;
    const cudaError_t e = kPairs[in][out].launch(plan, x, y, rows, static_cast<int>(cols), aligned,
                                                 period, offset, ctl,
                                                 reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? OS_OK : OS_ERR_CUDA;
}

}  // namespace

extern "C" {

const char* os_status_string(os_status s) {
    switch (s) {
        case OS_OK: return "OS_OK";
        case OS_ERR_NULL: return "OS_ERR_NULL: a required pointer is NULL";
        case OS_ERR_SHAPE: return "OS_ERR_SHAPE: a size or head dimension outside its range";
        case OS_ERR_DTYPE: return "OS_ERR_DTYPE: unknown dtype";
        case OS_ERR_K: return "OS_ERR_K: K outside [1, min(cols, 256)]";
        case OS_ERR_ALIAS: return "OS_ERR_ALIAS: an output overlaps an input or another output";
        case OS_ERR_CUDA: return "OS_ERR_CUDA: the CUDA runtime reported an error";
        case OS_ERR_TIMEOUT: return "OS_ERR_TIMEOUT: a device-side bounded wait gave up";
        case OS_ERR_PATH: return "OS_ERR_PATH: the kernel family cannot run this shape";
        case OS_ERR_ALIGN: return "OS_ERR_ALIGN: pointer not aligned to its element size";
        case OS_ERR_VALUE: return "OS_ERR_VALUE: a scalar argument outside its range";
    }
    return "unknown os_status";
}

os_status os_softmax_plan(int64_t rows, int64_t cols, os_dtype in, os_dtype out, os_path path,
                          os_plan* plan) {
    const os_status st = softmax_checks(rows, cols, in, out, path);
    if (st != OS_OK) return st;
    if (!plan) return OS_ERR_NULL;
    return kPairs[in][out].plan(rows, cols, path, true, plan);
}

os_status os_softmax_fwd_path(const void* x, void* y, int64_t rows, int64_t cols, os_dtype in,
                              os_dtype out, os_path path, os_stream_t stream) {
    return softmax_entry(x, y, rows, cols, in, out, path, 0, 0, stream);
}

os_status os_softmax_causal_fwd(const void* x, void* y, int64_t rows, int64_t cols,
                                int64_t period, int64_t offset, os_dtype in, os_dtype out,
                                os_stream_t stream) {
    if (period < 1 || offset < 0) return OS_ERR_SHAPE;
    return softmax_entry(x, y, rows, cols, in, out, OS_PATH_AUTO, period, offset, stream);
}

os_status os_softmax_stats(const void* x, float* m, float* d, float* lse, int64_t rows,
                           int64_t cols, os_dtype in, os_stream_t stream) {
    if (!valid_dtype(in)) return OS_ERR_DTYPE;
    if (!shape_ok(rows, cols)) return OS_ERR_SHAPE;
    if (rows == 0) return OS_OK;
    if (!x || (!m && !d && !lse)) return OS_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(x) % elem_bytes(in) || reinterpret_cast<uintptr_t>(m) % 4 ||
        reinterpret_cast<uintptr_t>(d) % 4 || reinterpret_cast<uintptr_t>(lse) % 4)
        return OS_ERR_ALIGN;
    const int64_t xb = rows * cols * elem_bytes(in), ob = rows * 4;
    const float* outs[3] = {m, d, lse};
    for (int i = 0; i < 3; ++i) {
        if (!outs[i]) continue;
        if (overlaps(x, xb, outs[i], ob)) return OS_ERR_ALIAS;
        for (int j = i + 1; j < 3; ++j)
            if (outs[j] && overlaps(outs[i], ob, outs[j], ob)) return OS_ERR_ALIAS;
    }
    const bool aligned = reinterpret_cast<uintptr_t>(x) % 16 == 0 && cols % elems_per_vector(in) == 0;
    if (!os::device_info()) return OS_ERR_CUDA;
    const cudaError_t e = os::launch_stats(x, in, m, d, lse, rows, static_cast<int>(cols), aligned,
                                           reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? OS_OK : OS_ERR_CUDA;
}

os_status os_softmax_fwd(const void* x, void* y, int64_t rows, int64_t cols, os_dtype in,
                         os_dtype out, os_stream_t stream) {
    return os_softmax_fwd_path(x, y, rows, cols, in, out, OS_PATH_AUTO, stream);
}

os_status os_topk_plan(int64_t rows, int64_t cols, int32_t K, os_plan* plan) {
    const os_status st = topk_checks(rows, cols, K);
    if (st != OS_OK) return st;
    if (!plan) return OS_ERR_NULL;
    return os::plan_topk(rows, cols, K, plan);
}

static os_status topk_entry(const float* x, float* vals, int32_t* idx, int64_t rows, int64_t cols,
                     int32_t K, bool plain, os_stream_t stream) {
    os_status st = topk_checks(rows, cols, K);
    if (st != OS_OK) return st;
    if (rows == 0) return OS_OK;
    if (!x || !vals || !idx) return OS_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(x) % 4 || reinterpret_cast<uintptr_t>(vals) % 4 ||
        reinterpret_cast<uintptr_t>(idx) % 4)
        return OS_ERR_ALIGN;
    const int64_t xb = rows * cols * 4, ob = rows * int64_t(K) * 4;
    if (overlaps(x, xb, vals, ob) || overlaps(x, xb, idx, ob) || overlaps(vals, ob, idx, ob))
        return OS_ERR_ALIAS;
    os_plan plan;
    st = os::plan_topk(rows, cols, K, &plan);
    if (st != OS_OK) return st;
    os::KernelCtl ctl;
    if (!make_ctl(&ctl)) return OS_ERR_CUDA;
    const cudaError_t e = os::launch_topk(plan, x, vals, idx, rows, static_cast<int>(cols), K, plain,
                                          ctl, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? OS_OK : OS_ERR_CUDA;
}

os_status os_softmax_topk(const float* x, float* vals, int32_t* idx, int64_t rows, int64_t cols,
                          int32_t K, os_stream_t stream) {
    return topk_entry(x, vals, idx, rows, cols, K, false, stream);
}

os_status os_topk(const float* x, float* vals, int32_t* idx, int64_t rows, int64_t cols, int32_t K,
                  os_stream_t stream) {
    return topk_entry(x, vals, idx, rows, cols, K, true, stream);
}

os_status os_topk_sample(const float* vals, const int32_t* idx, const float* u, int32_t* out,
                         int64_t rows, int32_t K, os_stream_t stream) {
    if (rows < 0) return OS_ERR_SHAPE;
    if (K < 1 || K > 256) return OS_ERR_K;
    if (rows > INT64_MAX / 8 / K) return OS_ERR_SHAPE;
    if (rows == 0) return OS_OK;
    if (!vals || !idx || !u || !out) return OS_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(vals) % 4 || reinterpret_cast<uintptr_t>(idx) % 4 ||
        reinterpret_cast<uintptr_t>(u) % 4 || reinterpret_cast<uintptr_t>(out) % 4)
        return OS_ERR_ALIGN;
    const int64_t kb = rows * int64_t(K) * 4, rb = rows * 4;
    if (overlaps(out, rb, vals, kb) || overlaps(out, rb, idx, kb) || overlaps(out, rb, u, rb))
        return OS_ERR_ALIAS;
    const cudaError_t e = os::launch_topk_sample(vals, idx, u, out, rows, K,
                                                 reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? OS_OK : OS_ERR_CUDA;
}

os_status os_attention_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                           int64_t bh, int64_t n, int32_t head_dim, float scale, int32_t causal,
                           os_stream_t stream) {
    if (bh < 0 || n < 0 || n > INT32_MAX || (head_dim != 64 && head_dim != 128))
        return OS_ERR_SHAPE;
    if (!(scale > 0.f) || !(scale < INFINITY) || (causal != 0 && causal != 1)) return OS_ERR_VALUE;
    if (bh == 0 || n == 0) return OS_OK;
    const int64_t nq = (n + 127) / 128;
    if (bh > INT32_MAX / nq || bh > INT64_MAX / 2 / head_dim / n) return OS_ERR_SHAPE;
    if (!q || !k || !v || !o) return OS_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(q) % 16 || reinterpret_cast<uintptr_t>(k) % 16 ||
        reinterpret_cast<uintptr_t>(v) % 16 || reinterpret_cast<uintptr_t>(o) % 16 ||
        reinterpret_cast<uintptr_t>(lse) % 4)
        return OS_ERR_ALIGN;
    const int64_t tb = bh * n * head_dim * 2, lb = bh * n * 4;
    if (overlaps(o, tb, q, tb) || overlaps(o, tb, k, tb) || overlaps(o, tb, v, tb))
        return OS_ERR_ALIAS;
    if (lse && (overlaps(lse, lb, q, tb) || overlaps(lse, lb, k, tb) || overlaps(lse, lb, v, tb) ||
                overlaps(lse, lb, o, tb)))
        return OS_ERR_ALIAS;
    os::KernelCtl ctl;
    if (!make_ctl(&ctl)) return OS_ERR_CUDA;
    const cudaError_t e = os::launch_attention(q, k, v, o, lse, bh, static_cast<int>(n), head_dim,
                                               scale, causal != 0, ctl,
                                               reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? OS_OK : OS_ERR_CUDA;
}

os_status os_attention_bwd(const void* q, const void* k, const void* v, const void* o,
                           const float* lse, const void* dout, const float* dlse, void* dq,
                           void* dk, void* dv, float* delta, int64_t bh, int64_t n,
                           int32_t head_dim, float scale, int32_t causal, os_stream_t stream) {
    if (bh < 0 || n < 0 || n > INT32_MAX || (head_dim != 64 && head_dim != 128))
        return OS_ERR_SHAPE;
    if (!(scale > 0.f) || !(scale < INFINITY) || (causal != 0 && causal != 1)) return OS_ERR_VALUE;
    if (bh == 0 || n == 0) return OS_OK;
    const int64_t nt = (n + 127) / 128;
    if (bh > INT32_MAX / nt || bh > INT64_MAX / 2 / head_dim / n) return OS_ERR_SHAPE;
    if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv || !delta) return OS_ERR_NULL;
    const int64_t tb = bh * n * head_dim * 2, lb = bh * n * 4;
    const struct {
        const void* p;
        int64_t bytes;
        int align;
    } in[] = {{q, tb, 16}, {k, tb, 16}, {v, tb, 16}, {o, tb, 16}, {dout, tb, 16}, {lse, lb, 4},
              {dlse, lb, 4}},
      out[] = {{dq, tb, 16}, {dk, tb, 16}, {dv, tb, 16}, {delta, lb, 4}};
    for (const auto& a : in)
        if (reinterpret_cast<uintptr_t>(a.p) % a.align) return OS_ERR_ALIGN;
    for (const auto& a : out)
        if (reinterpret_cast<uintptr_t>(a.p) % a.align) return OS_ERR_ALIGN;
    for (int i = 0; i < 4; ++i) {
        for (const auto& a : in)
            if (a.p && overlaps(out[i].p, out[i].bytes, a.p, a.bytes)) return OS_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return OS_ERR_ALIAS;
    }
    os::KernelCtl ctl;
    if (!make_ctl(&ctl)) return OS_ERR_CUDA;
    os::AttentionBwdArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.o = o;
    a.dout = dout;
    a.lse = lse;
    a.dlse = dlse;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.delta = delta;
    a.bh = bh;
    a.n = static_cast<int>(n);
    a.scale = scale;
    a.causal = causal != 0;
    const cudaError_t e = os::launch_attention_bwd(a, head_dim, ctl,
                                                   reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? OS_OK : OS_ERR_CUDA;
}

// Checks that the router and its gradient share.
static os_status route_checks(int64_t rows, int64_t experts, int32_t K, int64_t most_k,
                              os_score score, int32_t renorm, float scale, os_dtype in) {
    if (!valid_dtype(in)) return OS_ERR_DTYPE;
    if (rows < 0 || experts < 1 || experts > 1024 || rows > INT64_MAX / 8 / experts)
        return OS_ERR_SHAPE;
    if (K < 1 || K > 32 || K > most_k) return OS_ERR_K;
    if ((score != OS_SCORE_SOFTMAX && score != OS_SCORE_SIGMOID) || (renorm != 0 && renorm != 1) ||
        !(scale > -INFINITY) || !(scale < INFINITY))
        return OS_ERR_VALUE;
    return OS_OK;
}

os_status os_route_topk(const void* x, const float* bias, float* weights, int32_t* idx,
                        int64_t rows, int64_t experts, int32_t K, int32_t groups,
                        int32_t topk_groups, int32_t group_top, os_score score, int32_t renorm,
                        float scale, os_dtype in, os_stream_t stream) {
    if (experts < 1 || groups < 1 || groups > 32 || experts % groups || topk_groups < 1 ||
        topk_groups > groups || group_top < 1 || group_top > 2 || group_top > experts / groups)
        return OS_ERR_SHAPE;
    const os_status st = route_checks(rows, experts, K, experts / groups * topk_groups, score,
                                      renorm, scale, in);
    if (st != OS_OK) return st;
    if (rows == 0) return OS_OK;
    if (!x || !weights || !idx) return OS_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(x) % elem_bytes(in) || reinterpret_cast<uintptr_t>(bias) % 4 ||
        reinterpret_cast<uintptr_t>(weights) % 4 || reinterpret_cast<uintptr_t>(idx) % 4)
        return OS_ERR_ALIGN;
    const int64_t xb = rows * experts * elem_bytes(in), kb = rows * int64_t(K) * 4;
    if (overlaps(weights, kb, x, xb) || overlaps(idx, kb, x, xb) || overlaps(weights, kb, idx, kb) ||
        (bias && (overlaps(weights, kb, bias, experts * 4) || overlaps(idx, kb, bias, experts * 4))))
        return OS_ERR_ALIAS;
    os::RouteArgs a = {x, in, bias, rows, static_cast<int>(experts), K, groups, topk_groups,
                       group_top, score, renorm != 0, scale};
    const auto launch = in == OS_F32 ? os::route_fwd_f32 : os::route_fwd_bf16;
    const cudaError_t e = launch(a, weights, idx, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? OS_OK : OS_ERR_CUDA;
}

os_status os_route_bwd(const void* x, const int32_t* idx, const float* dweights, void* dx,
                       int64_t rows, int64_t experts, int32_t K, os_score score, int32_t renorm,
                       float scale, os_dtype in, os_stream_t stream) {
    const os_status st = route_checks(rows, experts, K, experts, score, renorm, scale, in);
    if (st != OS_OK) return st;
    if (rows == 0) return OS_OK;
    if (!x || !idx || !dweights || !dx) return OS_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(x) % elem_bytes(in) ||
        reinterpret_cast<uintptr_t>(dx) % elem_bytes(in) || reinterpret_cast<uintptr_t>(idx) % 4 ||
        reinterpret_cast<uintptr_t>(dweights) % 4)
        return OS_ERR_ALIGN;
    const int64_t xb = rows * experts * elem_bytes(in), kb = rows * int64_t(K) * 4;
    if (overlaps(dx, xb, x, xb) || overlaps(dx, xb, idx, kb) || overlaps(dx, xb, dweights, kb))
        return OS_ERR_ALIAS;
    os::RouteArgs a = {x, in, nullptr, rows, static_cast<int>(experts), K, 1, 1, 1, score,
                       renorm != 0, scale};
    const auto launch = in == OS_F32 ? os::route_bwd_f32 : os::route_bwd_bf16;
    const cudaError_t e = launch(a, idx, dweights, dx, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? OS_OK : OS_ERR_CUDA;
}

os_status os_sample(const void* x, const float* u, const os_sampling* s, int32_t* out, float* prob,
                    int64_t rows, int64_t cols, os_dtype in, os_stream_t stream) {
    if (!valid_dtype(in)) return OS_ERR_DTYPE;
    if (!shape_ok(rows, cols)) return OS_ERR_SHAPE;
    if (!s) return OS_ERR_NULL;
    if ((!s->temperature && !(s->temperature_all >= 0.f && s->temperature_all < INFINITY)) ||
        (!s->top_k && s->top_k_all < 0) ||
        (!s->top_p && !(s->top_p_all >= 0.f && s->top_p_all <= 1.f)) ||
        (!s->min_p && !(s->min_p_all >= 0.f && s->min_p_all <= 1.f)))
        return OS_ERR_VALUE;
    if (rows == 0) return OS_OK;
    if (!x || !u || !out) return OS_ERR_NULL;
    const void* words[] = {u, s->temperature, s->top_k, s->top_p, s->min_p};
    if (reinterpret_cast<uintptr_t>(x) % elem_bytes(in) || reinterpret_cast<uintptr_t>(out) % 4 ||
        reinterpret_cast<uintptr_t>(prob) % 4)
        return OS_ERR_ALIGN;
    for (const void* p : words)
        if (reinterpret_cast<uintptr_t>(p) % 4) return OS_ERR_ALIGN;
    const int64_t xb = rows * cols * elem_bytes(in), rb = rows * 4;
    if (prob && overlaps(out, rb, prob, rb)) return OS_ERR_ALIAS;
    for (const void* o : {static_cast<const void*>(out), static_cast<const void*>(prob)}) {
        if (!o) continue;
        if (overlaps(o, rb, x, xb)) return OS_ERR_ALIAS;
        for (const void* p : words)
            if (p && overlaps(o, rb, p, rb)) return OS_ERR_ALIAS;
    }
    const cudaError_t e = os::launch_sample(x, in, u, out, prob, rows, static_cast<int>(cols), *s,
                                            reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? OS_OK : OS_ERR_CUDA;
}

// Sizes of a paged cache, with `heads` query or key heads and `layers` copies of the pool.
static os_status paged_checks(const os_paged_cache* c, int64_t heads, int64_t layers) {
    if (!c) return OS_ERR_NULL;
    if (c->pages < 1 || c->seqs < 0 || c->width < 1 || c->kv_heads < 1 || c->page_size < 1 ||
        (c->head_dim != 64 && c->head_dim != 128) || heads < c->kv_heads || layers < 1)
        return OS_ERR_SHAPE;
    // (the kernels count a token's and a page's 16-byte pieces in 32 bits)
    if (c->kv_heads > (1 << 20) || c->page_size > (1 << 24)) return OS_ERR_SHAPE;
    if (c->pages > INT32_MAX / c->kv_heads / c->page_size || c->width > INT32_MAX / c->page_size ||
        c->seqs > INT32_MAX / heads || c->seqs > INT32_MAX / c->kv_heads / layers ||
        c->width > INT64_MAX / 8 / (c->seqs + 1))
        return OS_ERR_SHAPE;
    return OS_OK;
}

static os_status paged_pointers(const os_paged_cache* c) {
    if (!c->k || !c->v || !c->table || !c->lengths) return OS_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(c->k) % 16 || reinterpret_cast<uintptr_t>(c->v) % 16 ||
        reinterpret_cast<uintptr_t>(c->table) % 4 || reinterpret_cast<uintptr_t>(c->lengths) % 4)
        return OS_ERR_ALIGN;
    return OS_OK;
}

static int64_t pool_bytes(const os_paged_cache* c) {
    return c->pages * c->kv_heads * c->page_size * c->head_dim * 2;
}

// Rows of `row` elements `stride` apart: dense 16-byte pieces, no row over the next.
static bool rows_ok(int64_t rows, int64_t stride, int64_t row) {
    return stride >= row && stride % 8 == 0 && stride <= INT64_MAX / 4 / (rows + 1);
}

static int64_t rows_bytes(int64_t rows, int64_t stride, int64_t row) {
    return ((rows - 1) * stride + row) * 2;
}

os_status os_paged_append(const os_paged_cache* cache, const void* k, int64_t k_stride,
                          const void* v, int64_t v_stride, const void* q, int64_t q_stride,
                          void* q_out, const int32_t* starts, const float* inv_freq,
                          int64_t tokens, int32_t q_heads, int32_t rot, int32_t interleaved,
                          os_stream_t stream) {
    const os_status st = paged_checks(cache, q ? q_heads : cache ? cache->kv_heads : 1, 1);
    if (st != OS_OK) return st;
    const int64_t d = cache->head_dim, kv_row = cache->kv_heads * d, q_row = q ? q_heads * d : 0;
    if (tokens < 0 || tokens > INT32_MAX || (!starts && tokens != cache->seqs)) return OS_ERR_SHAPE;
    if (!rows_ok(tokens, k_stride, kv_row) || !rows_ok(tokens, v_stride, kv_row) ||
        (q && !rows_ok(tokens, q_stride, q_row)) || (q && q_heads > INT32_MAX / 2 / d) ||
        (inv_freq && (rot < 16 || rot > d || rot % 16)))
        return OS_ERR_SHAPE;
    if (interleaved != 0 && interleaved != 1) return OS_ERR_VALUE;
    if (tokens == 0 || cache->seqs == 0) return OS_OK;
    const os_status ps = paged_pointers(cache);
    if (ps != OS_OK) return ps;
    if (!k || !v || (q && !q_out) || (!q && q_out)) return OS_ERR_NULL;
    for (const void* p : {k, v, q, static_cast<const void*>(q_out)})
        if (reinterpret_cast<uintptr_t>(p) % 16) return OS_ERR_ALIGN;
    if (reinterpret_cast<uintptr_t>(starts) % 4 || reinterpret_cast<uintptr_t>(inv_freq) % 4)
        return OS_ERR_ALIGN;
    const Buffer written[] = {{cache->k, pool_bytes(cache)},
                              {cache->v, pool_bytes(cache)},
                              {q_out, tokens * q_row * 2}};
    const Buffer read[] = {{cache->table, cache->seqs * cache->width * 4},
                           {cache->lengths, cache->seqs * 4},
                           {k, rows_bytes(tokens, k_stride, kv_row)},
                           {v, rows_bytes(tokens, v_stride, kv_row)},
                           {q, rows_bytes(tokens, q_stride, q_row)},
                           {starts, (cache->seqs + 1) * 4},
                           {inv_freq, rot * 2}};
    if (!apart(written, read)) return OS_ERR_ALIAS;
    const os::PagedAppendArgs a = {q,        k,      v,       q_stride, k_stride, v_stride,        q_out,
                                   starts,   inv_freq, tokens, q_heads,  rot,      interleaved != 0};
    const cudaError_t e =
        os::launch_paged_append(*cache, a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? OS_OK : OS_ERR_CUDA;
}

os_status os_paged_attention_workspace(int64_t* bytes) {
    if (!bytes) return OS_ERR_NULL;
    const os::DeviceInfo* dev = os::device_info();
    if (!dev) return OS_ERR_CUDA;
    *bytes = os::paged_attention_workspace(dev->sms);
    return OS_OK;
}

os_status os_paged_attention(const os_paged_cache* cache, const void* q, int64_t q_stride,
                             void* out, float* lse, void* workspace, int32_t q_heads, float scale,
                             os_stream_t stream) {
    const os_status st = paged_checks(cache, q_heads, 1);
    if (st != OS_OK) return st;
    const int64_t row = int64_t(q_heads) * cache->head_dim;
    if (q_heads % cache->kv_heads || q_heads > INT32_MAX / 2 / cache->head_dim ||
        !rows_ok(cache->seqs, q_stride, row))
        return OS_ERR_SHAPE;
    // blocks of 16 keys that there can be, for 8 query heads each
    const int64_t units = int64_t(cache->kv_heads) * ((q_heads / cache->kv_heads + 7) / 8);
    const int64_t blocks = (cache->width * cache->page_size + 15) / 16;
    if (cache->seqs > 0 && units * blocks > (1 << 30) / cache->seqs) return OS_ERR_SHAPE;
    // (scores are formed as powers of two: scale log2 e has to be a number too)
    if (!(scale > 0.f) || !(scale * os::kScoreLog2e < INFINITY)) return OS_ERR_VALUE;
    if (cache->seqs == 0) return OS_OK;
    const os_status ps = paged_pointers(cache);
    if (ps != OS_OK) return ps;
    if (!q || !out || !workspace) return OS_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(q) % 16 || reinterpret_cast<uintptr_t>(out) % 16 ||
        reinterpret_cast<uintptr_t>(workspace) % 16 || reinterpret_cast<uintptr_t>(lse) % 4)
        return OS_ERR_ALIGN;
    const Buffer written[] = {{out, cache->seqs * row * 2}, {lse, cache->seqs * q_heads * 4}};
    const Buffer read[] = {{cache->k, pool_bytes(cache)},
                           {cache->v, pool_bytes(cache)},
                           {cache->table, cache->seqs * cache->width * 4},
                           {cache->lengths, cache->seqs * 4},
                           {q, rows_bytes(cache->seqs, q_stride, row)}};
    if (!apart(written, read)) return OS_ERR_ALIAS;
    int64_t wb = 0;
    const os_status ws = os_paged_attention_workspace(&wb);
    if (ws != OS_OK) return ws;
    const Buffer scratch[] = {{workspace, wb}};
    if (!apart(scratch, read) || !apart(scratch, written)) return OS_ERR_ALIAS;
    const cudaError_t e =
        os::launch_paged_attention(*cache, q, q_stride, out, lse, workspace, q_heads, scale,
                                   reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? OS_OK : OS_ERR_CUDA;
}

os_status os_paged_reorder(const os_paged_cache* cache, const int32_t* parents, int32_t* out_table,
                           int32_t* out_lengths, int32_t beams, int32_t layers,
                           os_stream_t stream) {
    const os_status st = paged_checks(cache, cache ? cache->kv_heads : 1, layers);
    if (st != OS_OK) return st;
    if (beams < 1 || cache->seqs % beams) return OS_ERR_SHAPE;
    if (pool_bytes(cache) > INT64_MAX / 4 / layers) return OS_ERR_SHAPE;
    if (cache->seqs == 0) return OS_OK;
    const os_status ps = paged_pointers(cache);
    if (ps != OS_OK) return ps;
    if (!parents || !out_table) return OS_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(parents) % 4 || reinterpret_cast<uintptr_t>(out_table) % 4 ||
        reinterpret_cast<uintptr_t>(out_lengths) % 4)
        return OS_ERR_ALIGN;
    const int64_t tb = cache->seqs * cache->width * 4, lb = cache->seqs * 4;
    const Buffer written[] = {{cache->k, pool_bytes(cache) * layers},
                              {cache->v, pool_bytes(cache) * layers},
                              {out_table, tb},
                              {out_lengths, lb}};
    const Buffer read[] = {{cache->table, tb}, {cache->lengths, lb}, {parents, lb}};
    if (!apart(written, read)) return OS_ERR_ALIAS;
    const cudaError_t e =
        os::launch_paged_reorder(*cache, parents, beams, layers, out_table, out_lengths,
                                 reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? OS_OK : OS_ERR_CUDA;
}

static os_status beam_checks(int64_t groups, int32_t beams, int64_t cols, int32_t K, os_dtype in) {
    if (!valid_dtype(in)) return OS_ERR_DTYPE;
    if (beams < 1 || beams > 64 || groups < 0 || groups > (1 << 26) / beams ||
        !shape_ok(groups * beams, cols))
        return OS_ERR_SHAPE;
    if (K < 1 || K > 64) return OS_ERR_K;
    return OS_OK;
}

os_status os_beam_select_workspace(int64_t groups, int32_t beams, int64_t cols, int32_t K,
                                   os_dtype in, int64_t* bytes) {
    const os_status st = beam_checks(groups, beams, cols, K, in);
    if (st != OS_OK) return st;
    if (!bytes) return OS_ERR_NULL;
    const os::DeviceInfo* dev = os::device_info();
    if (!dev) return OS_ERR_CUDA;
    *bytes = groups == 0 ? 0 : os::beam_select_workspace(groups, beams, cols, K, in, dev->sms);
    return OS_OK;
}

os_status os_beam_select(const void* x, const float* scores, const uint8_t* ended, float* out,
                         int32_t* parents, int32_t* tokens, void* workspace, int64_t groups,
                         int32_t beams, int64_t cols, int32_t K, int32_t pad, os_dtype in,
                         os_stream_t stream) {
    const os_status st = beam_checks(groups, beams, cols, K, in);
    if (st != OS_OK) return st;
    if (pad < 0 || pad >= cols) return OS_ERR_VALUE;
    if (groups == 0) return OS_OK;
    if (!x || !scores || !out || !parents || !tokens || !workspace) return OS_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(x) % elem_bytes(in) || reinterpret_cast<uintptr_t>(scores) % 4 ||
        reinterpret_cast<uintptr_t>(out) % 4 || reinterpret_cast<uintptr_t>(parents) % 4 ||
        reinterpret_cast<uintptr_t>(tokens) % 4 || reinterpret_cast<uintptr_t>(workspace) % 16)
        return OS_ERR_ALIGN;
    const int64_t rows = groups * beams, kb = groups * int64_t(K) * 4;
    const Buffer written[] = {{out, kb}, {parents, kb}, {tokens, kb}};
    const Buffer read[] = {{x, rows * cols * elem_bytes(in)}, {scores, rows * 4}, {ended, rows}};
    if (!apart(written, read)) return OS_ERR_ALIAS;
    int64_t wb = 0;
    const os_status ws = os_beam_select_workspace(groups, beams, cols, K, in, &wb);
    if (ws != OS_OK) return ws;
    const Buffer scratch[] = {{workspace, wb}};
    if (!apart(scratch, read) || !apart(scratch, written)) return OS_ERR_ALIAS;
    os::BeamSelectArgs a = {};
    a.x = x;
    a.in = in;
    a.scores = scores;
    a.ended = ended;
    a.out = out;
    a.parents = parents;
    a.tokens = tokens;
    a.workspace = workspace;
    a.groups = groups;
    a.cols = cols;
    a.beams = beams;
    a.K = K;
    a.pad = pad;
    const cudaError_t e = os::launch_beam_select(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? OS_OK : OS_ERR_CUDA;
}

os_status os_exp_f32(const float* z, float* out, int64_t n, os_stream_t stream) {
    if (n < 0) return OS_ERR_SHAPE;
    if (n == 0) return OS_OK;
    if (!z || !out) return OS_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(z) % 4 || reinterpret_cast<uintptr_t>(out) % 4)
        return OS_ERR_ALIGN;
    const cudaError_t e = os::launch_exp(z, out, n, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? OS_OK : OS_ERR_CUDA;
}

static os_status exp_pairs_entry(const float* z, float* out, int64_t n, int degree, os_stream_t stream) {
    if (n < 0) return OS_ERR_SHAPE;
    if (n == 0) return OS_OK;
    if (!z || !out) return OS_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(z) % 4 || reinterpret_cast<uintptr_t>(out) % 4)
        return OS_ERR_ALIGN;
    const cudaError_t e = os::launch_exp_pairs(z, out, n, degree,
                                               reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? OS_OK : OS_ERR_CUDA;
}

os_status os_exp_pairs_f32(const float* z, float* out, int64_t n, os_stream_t stream) {
    return exp_pairs_entry(z, out, n, 5, stream);
}

os_status os_exp_pairs_coarse_f32(const float* z, float* out, int64_t n, os_stream_t stream) {
    return exp_pairs_entry(z, out, n, 3, stream);
}

os_status os_device_status(os_stream_t stream) {
    if (!status_word()) return OS_ERR_CUDA;
    // one host caller at a time per process: the exchange's result word is shared
    static std::mutex mu;
    std::lock_guard<std::mutex> lock(mu);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    status_exchange_kernel<<<1, 1, 0, s>>>();
    if (cudaGetLastError() != cudaSuccess) return OS_ERR_CUDA;
    unsigned int v = 0;
    if (cudaMemcpyFromSymbolAsync(&v, os_device_status_taken, sizeof(v), 0,
                                  cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return OS_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return OS_ERR_CUDA;
    if (v == 0) return OS_OK;
    return (v & os::kErrWaitTimeout) ? OS_ERR_TIMEOUT : OS_ERR_CUDA;
}

os_status os_set_wait_timeout_ns(uint64_t ns) {
    if (ns < 1000000ull || ns > 10000000000ull) return OS_ERR_SHAPE;
    g_timeout_ns.store(ns);
    return OS_OK;
}

os_status os_set_fault_injection(int32_t mode) {
    if (mode != 0 && mode != os::kFaultSkipFirstLoad) return OS_ERR_SHAPE;
    g_fault.store(mode);
    return OS_OK;
}

}  // extern "C"
