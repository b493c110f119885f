// library.cu -- the one translation unit of libfp8q.so: the quantisers and GEMMs (fp8q.cu), and the
// C entry points of the routed expert layer's operators (kernels in moe.cuh).  One unit, so that all
// kernels share the device status word and the launch helpers.
#include <cmath>

#include "fp8q.cu"

#include "moe.cuh"

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int64_t kI32 = 0x7FFFFFFF;

// Division of n < 2^31 by d as (umulhi(n, mul) + n) >> shift: with 2^shift the smallest power of two not
// below d, mul = floor(2^32 (2^shift - d) / d) + 1 (Granlund and Montgomery, "Division by invariant
// integers using multiplication", 1994).
FastDiv fast_div(uint32_t d)
{
    uint32_t shift = 0;
    while ((1ull << shift) < d) ++shift;
    return FastDiv{(uint32_t)(((1ull << 32) * ((1ull << shift) - d)) / d + 1), shift};
}

// A persistent grid: `per_sm` CTAs on each SM, no more than there are work items.
unsigned grid_for(int64_t items, int per_sm)
{
    int sms = sm_count();
    if (sms <= 0) sms = 148;
    const int64_t n = (int64_t)sms * per_sm;
    return (unsigned)(items < n ? (items > 0 ? items : 1) : n);
}

// One cluster of `ctas` CTAs, in programmatic stream order as launch_kernel.
template <typename... KArgs, typename... Args>
int launch_cluster(void (*kern)(KArgs...), int ctas, dim3 block, size_t smem, cudaStream_t st, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess) return launch_status();
    cudaGetLastError();
    if (cfg.numAttrs == 1) return FP8Q_ERR_CUDA;
    cfg.numAttrs = 1;   // the driver refused the combination: launch in plain stream order
    if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
        cudaGetLastError();
        return FP8Q_ERR_CUDA;
    }
    return launch_status();
}

// One CTA does this many slots as fast as a cluster starts and meets: 8 slots 3.1 us against 4.5, 1024
// slots 4.8 against 5.1, 4096 slots 8.8 against 6.3.
constexpr int64_t kPlanOneCta = 1024;

// Lets a kernel have up to `bytes` of dynamic shared memory, once a device (`ready`: the kernel's own).
template <typename Kernel>
bool allow_smem(Kernel kern, int bytes, std::atomic<bool> (&ready)[kMaxDevices])
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
    if (ready[dev].load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    ready[dev].store(true, std::memory_order_release);
    return true;
}

// s where n = 2^s nv, -1 where there is none.
int lane_shift(int n, int nv)
{
    for (int s = 0; s < 6; ++s)
        if (n == nv << s) return s;
    return -1;
}

template <typename L, bool SOFTMAX>
int launch_route(const void* logits, const float* bias, int64_t T, int E, int k, int n_group, int topk_group,
                 int renorm, float scale, int32_t* idx, float* w, cudaStream_t st)
{
    const dim3 grid((unsigned)((T + 3) / 4));
    const L* l = static_cast<const L*>(logits);
    const int per = E / n_group;
    const bool wide = E % 8 == 0 && aligned16(logits) && aligned16(bias);
#define FP8Q_ROUTE(NV)                                                                                             \
    return launch_kernel(moe_route_kernel<L, NV, SOFTMAX>, grid, dim3(128), 0, st, false, l, bias, T,              \
                         RouteShape{E, k, n_group, topk_group, per, lane_shift(per, NV)}, wide, renorm, scale, idx, w)
    if (E <= 32) FP8Q_ROUTE(1);
    if (E <= 64) FP8Q_ROUTE(2);
    if (E <= 128) FP8Q_ROUTE(4);
    if (E <= 256) FP8Q_ROUTE(8);
    if (E <= 512) FP8Q_ROUTE(16);
    FP8Q_ROUTE(32);
#undef FP8Q_ROUTE
}

template <typename L, bool DENSE>
int launch_route_backward(const float* dw, const float* w, const int32_t* idx, const void* logits, int64_t T, int E,
                          int k, int sigmoid, int renorm, float scale, void* dlogits, cudaStream_t st)
{
    const dim3 grid((unsigned)((T + 3) / 4));
    const L* l = static_cast<const L*>(logits);
    L* d = static_cast<L*>(dlogits);
    const bool wide = E % 8 == 0 && aligned16(logits) && aligned16(dlogits);
#define FP8Q_ROUTE(NV)                                                                                             \
    return launch_kernel(moe_route_backward_kernel<L, NV, DENSE>, grid, dim3(128), 0, st, false, dw, w, idx, l, T, E, \
                         k, wide, sigmoid, renorm, scale, d)
    if (E <= 32) FP8Q_ROUTE(1);
    if (E <= 64) FP8Q_ROUTE(2);
    if (E <= 128) FP8Q_ROUTE(4);
    if (E <= 256) FP8Q_ROUTE(8);
    if (E <= 512) FP8Q_ROUTE(16);
    FP8Q_ROUTE(32);
#undef FP8Q_ROUTE
}

// What both directions of the router ask of their scalar arguments.
int route_args(int logits_type, int64_t T, int32_t E, int32_t k, int score, float scale)
{
    if (T < 0 || E < 1 || k < 1 || k > E) return FP8Q_ERR_ARG;
    if (logits_type != FP8Q_LOGITS_FP32 && logits_type != FP8Q_LOGITS_BF16) return FP8Q_ERR_ARG;
    if (score != FP8Q_SCORE_SIGMOID && score != FP8Q_SCORE_SOFTMAX) return FP8Q_ERR_ARG;
    if (!std::isfinite(scale) || scale == 0.0f) return FP8Q_ERR_ARG;
    if (E > kMoeMaxExperts || k > kMoeMaxTopK || T > kI32 / k) return FP8Q_ERR_UNSUPPORTED;
    return FP8Q_OK;
}

}  // namespace

extern "C" {

int fp8q_moe_route(const void* logits, int logits_type, const float* bias, int64_t T, int32_t E, int32_t k,
                   int32_t n_group, int32_t topk_group, int score, int renormalize, float scale, int32_t* idx,
                   float* w, fp8q_stream_t stream)
{
    const int rc = route_args(logits_type, T, E, k, score, scale);
    if (rc != FP8Q_OK) return rc;
    if (n_group < 1 || topk_group < 1 || topk_group > n_group || E % n_group != 0) return FP8Q_ERR_ARG;
    if ((int64_t)topk_group * (E / n_group) < k) return FP8Q_ERR_ARG;
    if (n_group > kMoeMaxGroups) return FP8Q_ERR_UNSUPPORTED;
    if (T == 0) return FP8Q_OK;
    if (!logits || !idx || !w) return FP8Q_ERR_ARG;
    const bool bf16 = logits_type == FP8Q_LOGITS_BF16;
    if ((reinterpret_cast<uintptr_t>(logits) & (bf16 ? 1u : 3u)) != 0 || !aligned4(bias) || !aligned4(idx) ||
        !aligned4(w))
        return FP8Q_ERR_ALIGN;
    const cudaStream_t st = (cudaStream_t)stream;
    const bool softmax = score == FP8Q_SCORE_SOFTMAX;
    const auto launch = bf16 ? (softmax ? launch_route<uint16_t, true> : launch_route<uint16_t, false>)
                             : (softmax ? launch_route<float, true> : launch_route<float, false>);
    return launch(logits, bias, T, E, k, n_group, topk_group, renormalize != 0, scale, idx, w, st);
}

int fp8q_moe_route_backward(const float* dw, const float* w, const int32_t* idx, const void* logits, int logits_type,
                            int64_t T, int32_t E, int32_t k, int score, int renormalize, float scale, void* dlogits,
                            fp8q_stream_t stream)
{
    const int rc = route_args(logits_type, T, E, k, score, scale);
    if (rc != FP8Q_OK) return rc;
    if (T == 0) return FP8Q_OK;
    if (!dw || !w || !idx || !logits || !dlogits) return FP8Q_ERR_ARG;
    const bool bf16 = logits_type == FP8Q_LOGITS_BF16;
    const uintptr_t both = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(dlogits);
    if ((both & (bf16 ? 1u : 3u)) != 0 || !aligned4(dw) || !aligned4(w) || !aligned4(idx)) return FP8Q_ERR_ALIGN;
    const cudaStream_t st = (cudaStream_t)stream;
    const bool sigmoid = score == FP8Q_SCORE_SIGMOID, dense = !sigmoid && renormalize == 0;
    const auto launch = bf16 ? (dense ? launch_route_backward<uint16_t, true> : launch_route_backward<uint16_t, false>)
                             : (dense ? launch_route_backward<float, true> : launch_route_backward<float, false>);
    return launch(dw, w, idx, logits, T, E, k, sigmoid, renormalize != 0, scale, dlogits, st);
}

int fp8q_moe_plan(const int32_t* idx, int64_t T, int32_t k, int32_t E, int32_t* offsets, int32_t* slots,
                  int32_t* rows, fp8q_stream_t stream)
{
    if (T < 0 || k < 1 || E < 1) return FP8Q_ERR_ARG;
    if (E > kMoeMaxExperts || k > kMoeMaxTopK || T > kI32 / k) return FP8Q_ERR_UNSUPPORTED;
    if (!offsets || (T > 0 && (!idx || !slots || !rows))) return FP8Q_ERR_ARG;
    if (!aligned4(idx) || !aligned4(offsets) || !aligned4(slots) || !aligned4(rows)) return FP8Q_ERR_ALIGN;
    const cudaStream_t st = (cudaStream_t)stream;
    if (T == 0) {
        const size_t bytes = (size_t)(E + 1) * sizeof(int32_t);
        return cudaMemsetAsync(offsets, 0, bytes, st) == cudaSuccess ? FP8Q_OK : FP8Q_ERR_CUDA;
    }
    const int ctas = T * k <= kPlanOneCta ? 1 : kPlanCtas;
    const auto plan = ctas == 1 ? moe_plan_kernel<1> : moe_plan_kernel<kPlanCtas>;
    static std::atomic<bool> ready[2][kMaxDevices];
    if (!allow_smem(plan, plan_smem(kMoeMaxExperts), ready[ctas == 1])) return FP8Q_ERR_CUDA;
    return launch_cluster(plan, ctas, dim3(kPlanThreads), (size_t)plan_smem(E), st, idx, T * k, (int)E, offsets, slots,
                          rows);
}

int fp8q_moe_dispatch(const uint16_t* x, const int32_t* offsets, const int32_t* slots, const int32_t* rows,
                      const float* weights, int32_t E, int64_t T, int32_t k, int64_t C, uint8_t* q, float* s,
                      uint8_t* qt, float* st, int64_t Kcap, fp8q_stream_t stream)
{
    if (T < 0 || k < 1 || E < 1 || C < 0 || Kcap < 0) return FP8Q_ERR_ARG;
    if (E > kMoeMaxExperts || k > kMoeMaxTopK || T > kI32 / k || C > kI32 || Kcap > kI32) return FP8Q_ERR_UNSUPPORTED;
    if (C % 128 != 0 || Kcap % 128 != 0) return FP8Q_ERR_SHAPE;
    if (T == 0 || C == 0) return FP8Q_OK;
    if (!x || !offsets || !slots || !rows || !q || !s || (qt == nullptr) != (st == nullptr)) return FP8Q_ERR_ARG;
    if (!aligned16(x) || !aligned16(q) || !aligned16(s) || !aligned16(qt) || !aligned16(st)) return FP8Q_ERR_ALIGN;
    if (!aligned4(offsets) || !aligned4(slots) || !aligned4(rows) || !aligned4(weights)) return FP8Q_ERR_ALIGN;
    const cudaStream_t cs = (cudaStream_t)stream;
    const int64_t M = T * k;
    const int64_t quads = T * ((C / 128 + 3) / 4), tiles = ((M + 127) / 128 + E) * (C / 128);
    if (quads > kI32 || tiles > kI32) return FP8Q_ERR_UNSUPPORTED;
    const auto by_row = weights ? moe_dispatch_rows_kernel<true> : moe_dispatch_rows_kernel<false>;
    const int done = launch_kernel(by_row, dim3(grid_for((quads + 7) / 8, 8)), dim3(256), qt ? group_table_bytes(E) : 0, cs,
                                   false, x, rows, weights, (uint32_t)T, (uint32_t)k, (uint32_t)C, q, s,
                                   qt ? offsets : nullptr, (int)E, Kcap);
    if (done != FP8Q_OK || !qt) return done;
    const int64_t items = ((M + 127) / 128 + E) * ((C / 128 + kColBlocks - 1) / kColBlocks);
    const auto by_column = weights ? moe_dispatch_cols_kernel<true> : moe_dispatch_cols_kernel<false>;
    static std::atomic<bool> ready[2][kMaxDevices];
    if (!allow_smem(by_column, gather_smem(kMoeMaxExperts), ready[weights != nullptr])) return FP8Q_ERR_CUDA;
    return launch_kernel(by_column, dim3(grid_for(items, 3)), dim3(256), gather_smem(E), cs, false, x, slots, weights,
                         offsets, (int)E, M, fast_div((uint32_t)k), (uint32_t)C, qt, st, Kcap);
}

int fp8q_moe_combine(const uint16_t* y, const int32_t* rows, const float* weights, const uint16_t* add, int64_t T,
                     int32_t k, int64_t C, uint16_t* out, fp8q_stream_t stream)
{
    if (T < 0 || k < 1 || C < 0) return FP8Q_ERR_ARG;
    if (k > kMoeMaxTopK || T > kI32 / k || C > kI32) return FP8Q_ERR_UNSUPPORTED;
    if (C % 8 != 0) return FP8Q_ERR_SHAPE;
    if (T == 0 || C == 0) return FP8Q_OK;
    if (!y || !rows || !out) return FP8Q_ERR_ARG;
    if (!aligned16(y) || !aligned16(add) || !aligned16(out) || !aligned4(rows) || !aligned4(weights))
        return FP8Q_ERR_ALIGN;
    const int64_t items = T * ((C / 8 + kCombineThreads - 1) / kCombineThreads);
    if (items > kI32) return FP8Q_ERR_UNSUPPORTED;
    return launch_kernel(moe_combine_kernel, dim3(grid_for(items, 8)), dim3(kCombineThreads), 0, (cudaStream_t)stream, false,
                         y, rows, weights, add, (uint32_t)T, (uint32_t)k, (uint32_t)C, out);
}

int fp8q_moe_combine_dweight(const uint16_t* dout, const uint16_t* y, const int32_t* rows, int64_t T, int32_t k,
                             int64_t C, float* dw, fp8q_stream_t stream)
{
    if (T < 0 || k < 1 || C < 0) return FP8Q_ERR_ARG;
    if (k > kMoeMaxTopK || T > kI32 / k || C > kI32) return FP8Q_ERR_UNSUPPORTED;
    if (C % 8 != 0) return FP8Q_ERR_SHAPE;
    if (T == 0) return FP8Q_OK;
    if (!dw || !rows || (C > 0 && (!dout || !y))) return FP8Q_ERR_ARG;
    if (!aligned16(dout) || !aligned16(y) || !aligned4(rows) || !aligned4(dw)) return FP8Q_ERR_ALIGN;
    return launch_kernel(moe_combine_dweight_kernel, dim3((unsigned)((T * k + 7) / 8)), dim3(256), 0,
                         (cudaStream_t)stream, false, dout, y, rows, T, (int)k, C, dw);
}

int fp8q_swiglu_quant(const uint16_t* h, int64_t M, int64_t I, uint8_t* q, float* s, uint8_t* hq, float* hs,
                      fp8q_stream_t stream)
{
    if (M < 0 || I < 0) return FP8Q_ERR_ARG;
    if (I % 128 != 0) return FP8Q_ERR_SHAPE;
    if (M == 0 || I == 0) return FP8Q_OK;
    if (M > kI32 || I > kI32 / 2) return FP8Q_ERR_UNSUPPORTED;
    if (!h || !q || !s || (hq == nullptr) != (hs == nullptr)) return FP8Q_ERR_ARG;
    if (!aligned16(h) || !aligned16(q) || !aligned16(s) || !aligned16(hq) || !aligned16(hs)) return FP8Q_ERR_ALIGN;
    // Eight rows a warp, or one where that leaves too few warps to cover the latency (16 fit an SM here).
    // I = 2048 with the checkpoint: 2048 rows 10.4 us with eight and 7.7 with one, 4096 rows 10.9 and 12.5.
    const int64_t quads = (I / 128 + 3) / 4;
    const int64_t rows = (M + 7) / 8 * quads >= 5 * (int64_t)grid_for(kI32, 2) ? 8 : 1;
    const int64_t items = (M + rows - 1) / rows * quads;
    if (items > kI32) return FP8Q_ERR_UNSUPPORTED;
    const auto kern = hq ? swiglu_quant_kernel<true> : swiglu_quant_kernel<false>;
    return launch_kernel(kern, dim3(grid_for((items + 7) / 8, 2)), dim3(256), 0, (cudaStream_t)stream, false, h,
                         (uint32_t)M, (uint32_t)I, (uint32_t)rows, q, s, hq, hs);
}

int fp8q_swiglu_backward_quant(const uint16_t* da, const uint8_t* hq, const float* hs, const int32_t* offsets,
                               int32_t E, int64_t M, int64_t I, uint8_t* q, float* s, uint8_t* qt, float* st,
                               uint8_t* aqt, float* ast, int64_t Kcap, fp8q_stream_t stream)
{
    if (M < 0 || I < 0 || E < 1 || Kcap < 0 || (!offsets && E != 1)) return FP8Q_ERR_ARG;
    if (I % 128 != 0 || Kcap % 128 != 0) return FP8Q_ERR_SHAPE;
    if (E > kMoeMaxExperts || M > kI32 || I > kI32 / 2 || Kcap > kI32) return FP8Q_ERR_UNSUPPORTED;
    if (M == 0 || I == 0) return FP8Q_OK;
    if (!da || !hq || !hs || !q || !s || !qt || !st || !aqt || !ast) return FP8Q_ERR_ARG;
    if (!offsets && Kcap < M) return FP8Q_ERR_SHAPE;
    if (!aligned16(da) || !aligned16(hq) || !aligned16(hs) || !aligned16(q) || !aligned16(s) || !aligned16(qt) ||
        !aligned16(st) || !aligned16(aqt) || !aligned16(ast) || !aligned4(offsets))
        return FP8Q_ERR_ALIGN;
    const int64_t tiles = ((M + 127) / 128 + E) * (I / 128);
    if (tiles > kI32) return FP8Q_ERR_UNSUPPORTED;
    static std::atomic<bool> ready[kMaxDevices];
    if (!allow_smem(swiglu_backward_kernel, back_smem(kMoeMaxExperts), ready)) return FP8Q_ERR_CUDA;
    return launch_kernel(swiglu_backward_kernel, dim3(grid_for(tiles, 1)), dim3(kBackThreads), back_smem(E),
                         (cudaStream_t)stream, false, da, hq, hs, offsets, (int)E, M, (uint32_t)I, q, s, qt, st, aqt, ast,
                         Kcap);
}

}  // extern "C"
