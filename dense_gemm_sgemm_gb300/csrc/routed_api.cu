// Host side of the routed products' C entry points: argument checks, then the launchers.
#include <cuda_runtime.h>

#include "routed_internal.h"

namespace gemm {
namespace {

constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxLd = int64_t(1) << 35;
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxDim24 = (int64_t(1) << 24) - 1;

bool is_type(int t) { return t == GEMM_TYPE_F32 || t == GEMM_TYPE_F16 || t == GEMM_TYPE_BF16; }
bool is_type16(int t) { return t == GEMM_TYPE_F16 || t == GEMM_TYPE_BF16; }
int size_of(int t) { return t == GEMM_TYPE_F32 ? 4 : 2; }
bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
// Index and weight arrays: 4-byte elements.
template <class... P> bool words(P... p) { return (aligned(p, 4) && ...); }
gemm_status_t from_cuda(cudaError_t e)
{
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}
gemm_status_t usable(DeviceInfo &dev)
{
    return current_device(dev) && dev.cc_major == 10 && dev.cc_minor == 3 ? GEMM_OK : GEMM_ERR_NO_DEVICE;
}
// A matrix of `cols` columns and its leading dimension.
bool ld_ok(int64_t ld, int64_t cols) { return ld >= (cols > 1 ? cols : 1); }

gemm_status_t check_choice(int64_t T, int64_t E, int top_k)
{
    if (T < 0 || E < 1 || top_k < 1 || top_k > E) return GEMM_ERR_INVALID_VALUE;
    if (E > 1024 || top_k > 32 || T > kMaxInt / (E > top_k ? E : top_k)) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

}  // namespace
}  // namespace gemm

using namespace gemm;

extern "C" {

gemm_status_t gemm_moe_route(gemm_type_t type, int64_t T, int64_t E, const void *logits, int64_t ld, const float *bias,
                             gemm_score_t score, int groups, int groups_kept, int group_top, int top_k,
                             int renormalise, float scale, int32_t *ids, float *weights, int32_t *offsets,
                             int32_t *tokens, int32_t *where, void *stream)
{
    if (!is_type(type) || (score != GEMM_SCORE_SOFTMAX && score != GEMM_SCORE_SIGMOID)) return GEMM_ERR_INVALID_VALUE;
    gemm_status_t s = check_choice(T, E, top_k);
    if (s != GEMM_OK) return s;
    if (groups < 1 || E % groups != 0 || groups_kept < 1 || groups_kept > groups || group_top < 1 || group_top > 2 ||
        top_k > E / groups * groups_kept || !ld_ok(ld, E))
        return GEMM_ERR_INVALID_VALUE;
    if (groups > 32 || ld > kMaxLd) return GEMM_ERR_UNSUPPORTED;
    const bool plan = offsets != nullptr;
    if (plan ? T > 0 && (tokens == nullptr || where == nullptr) : tokens != nullptr || where != nullptr)
        return GEMM_ERR_INVALID_VALUE;
    if (T > 0 && (logits == nullptr || ids == nullptr || weights == nullptr)) return GEMM_ERR_INVALID_VALUE;
    if (!aligned(logits, size_of(type)) || !words(bias, ids, weights, offsets, tokens, where)) return GEMM_ERR_MISALIGNED;
    if (T == 0 && !plan) return GEMM_OK;
    DeviceInfo dev;
    if ((s = usable(dev)) != GEMM_OK) return s;
    const RouteArgs a{type, T, int(E), logits, ld, bias, score, groups, groups_kept, group_top, top_k, renormalise != 0,
                      scale, ids, weights, offsets, tokens, where, false};
    return from_cuda(launch_route(a, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_moe_route_backward(gemm_type_t type, int64_t T, int64_t E, const float *dweights, const void *logits,
                                      int64_t ld, const int32_t *ids, gemm_score_t score, int top_k, int renormalise,
                                      float scale, void *dlogits, int64_t ldd, void *stream)
{
    if (!is_type(type) || (score != GEMM_SCORE_SOFTMAX && score != GEMM_SCORE_SIGMOID)) return GEMM_ERR_INVALID_VALUE;
    gemm_status_t s = check_choice(T, E, top_k);
    if (s != GEMM_OK) return s;
    if (!ld_ok(ld, E) || !ld_ok(ldd, E)) return GEMM_ERR_INVALID_VALUE;
    if (ld > kMaxLd || ldd > kMaxLd) return GEMM_ERR_UNSUPPORTED;
    if (T == 0) return GEMM_OK;
    if (dweights == nullptr || logits == nullptr || ids == nullptr || dlogits == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (!aligned(logits, size_of(type)) || !aligned(dlogits, size_of(type)) || !words(dweights, ids))
        return GEMM_ERR_MISALIGNED;
    DeviceInfo dev;
    if ((s = usable(dev)) != GEMM_OK) return s;
    RouteArgs a{};
    a.type = type;
    a.T = T;
    a.E = int(E);
    a.logits = logits;
    a.ld = ld;
    a.score = score;
    a.top_k = top_k;
    a.renormalise = renormalise != 0;
    a.scale = scale;
    return from_cuda(launch_route_backward(a, dweights, ids, dlogits, ldd, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_moe_plan(int64_t T, int64_t E, int top_k, const int32_t *ids, int32_t *offsets, int32_t *tokens,
                            int32_t *where, void *stream)
{
    // unlike a router's, given choices may name an expert more than once
    gemm_status_t s;
    if (T < 0 || E < 1 || top_k < 1) return GEMM_ERR_INVALID_VALUE;
    if (E > 1024 || top_k > 1024 || T > kMaxInt / top_k) return GEMM_ERR_UNSUPPORTED;
    if (offsets == nullptr || (T > 0 && (ids == nullptr || tokens == nullptr || where == nullptr)))
        return GEMM_ERR_INVALID_VALUE;
    if (!words(ids, offsets, tokens, where)) return GEMM_ERR_MISALIGNED;
    DeviceInfo dev;
    if ((s = usable(dev)) != GEMM_OK) return s;
    return from_cuda(launch_plan(T, int(E), top_k, ids, offsets, tokens, where, static_cast<cudaStream_t>(stream)));
}

static gemm_status_t check_rows(int64_t T, int64_t H, int top_k, int64_t positions)
{
    if (T < 0 || H < 0 || top_k < 1 || positions < 0) return GEMM_ERR_INVALID_VALUE;
    if (T > kMaxInt / top_k || H > kMaxDim24 || positions > kMaxInt || top_k > 1024) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

gemm_status_t gemm_moe_dispatch(gemm_type_t type, int64_t T, int64_t H, int top_k, const void *x, int64_t ldx,
                                const int32_t *where, const float *weights, int64_t positions, void *out, int64_t ldo,
                                void *stream)
{
    if (!is_type(type)) return GEMM_ERR_INVALID_VALUE;
    gemm_status_t s = check_rows(T, H, top_k, positions);
    if (s != GEMM_OK) return s;
    if (!ld_ok(ldx, H) || !ld_ok(ldo, H)) return GEMM_ERR_INVALID_VALUE;
    if (ldx > kMaxLd || ldo > kMaxLd) return GEMM_ERR_UNSUPPORTED;
    if (T == 0 || H == 0 || positions == 0) return GEMM_OK;
    if (x == nullptr || where == nullptr || out == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (!aligned(x, size_of(type)) || !aligned(out, size_of(type)) || !words(where, weights)) return GEMM_ERR_MISALIGNED;
    DeviceInfo dev;
    if ((s = usable(dev)) != GEMM_OK) return s;
    return from_cuda(launch_dispatch(type, GEMM_TYPE_F32, T, H, top_k, x, ldx, nullptr, 0, positions, where, weights, out,
                                     ldo, nullptr, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_moe_combine(gemm_type_t rows_type, gemm_type_t y_type, int64_t T, int64_t H, int top_k,
                               const void *rows, int64_t ldr, int64_t positions, const int32_t *where,
                               const float *weights, void *y, int64_t ldy, void *stream)
{
    if (!is_type(rows_type) || !is_type(y_type)) return GEMM_ERR_INVALID_VALUE;
    gemm_status_t s = check_rows(T, H, top_k, positions);
    if (s != GEMM_OK) return s;
    if (!ld_ok(ldr, H) || !ld_ok(ldy, H)) return GEMM_ERR_INVALID_VALUE;
    if (ldr > kMaxLd || ldy > kMaxLd) return GEMM_ERR_UNSUPPORTED;
    if (T == 0 || H == 0) return GEMM_OK;
    if ((rows == nullptr && positions > 0) || where == nullptr || y == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (!aligned(rows, size_of(rows_type)) || !aligned(y, size_of(y_type)) || !words(where, weights))
        return GEMM_ERR_MISALIGNED;
    DeviceInfo dev;
    if ((s = usable(dev)) != GEMM_OK) return s;
    return from_cuda(launch_combine(rows_type, y_type, T, H, top_k, rows, ldr, positions, where, weights, y, ldy,
                                    static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_moe_combine_backward(gemm_type_t type, gemm_type_t rows_type, int64_t T, int64_t H, int top_k,
                                        const void *dy, int64_t lddy, const void *rows, int64_t ldr, int64_t positions,
                                        const int32_t *where, const float *weights, void *drows, int64_t lddr,
                                        float *dweights, void *stream)
{
    if (!is_type(type) || !is_type(rows_type)) return GEMM_ERR_INVALID_VALUE;
    gemm_status_t s = check_rows(T, H, top_k, positions);
    if (s != GEMM_OK) return s;
    if (!ld_ok(lddy, H) || !ld_ok(ldr, H) || !ld_ok(lddr, H)) return GEMM_ERR_INVALID_VALUE;
    if (lddy > kMaxLd || ldr > kMaxLd || lddr > kMaxLd) return GEMM_ERR_UNSUPPORTED;
    if (T == 0) return GEMM_OK;
    if (where == nullptr || dweights == nullptr || (H > 0 && dy == nullptr) ||
        (H > 0 && positions > 0 && (rows == nullptr || drows == nullptr)))
        return GEMM_ERR_INVALID_VALUE;
    if (!aligned(dy, size_of(type)) || !aligned(drows, size_of(type)) || !aligned(rows, size_of(rows_type)) ||
        !words(where, weights, dweights))
        return GEMM_ERR_MISALIGNED;
    DeviceInfo dev;
    if ((s = usable(dev)) != GEMM_OK) return s;
    return from_cuda(launch_dispatch(type, rows_type, T, H, top_k, dy, lddy, rows, ldr, positions, where, weights, drows,
                                     lddr, dweights, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_gated_silu_backward(gemm_type_t type, gemm_type_t dh_type, int64_t rows, int64_t I, const void *pre,
                                       int64_t ldp, const void *dh, int64_t lddh, void *dpre, int64_t lddp, void *stream)
{
    if (!is_type16(type) || (dh_type != type && dh_type != GEMM_TYPE_F32) || rows < 0 || I < 0) return GEMM_ERR_INVALID_VALUE;
    if (rows > kMaxInt || I > kMaxDim24) return GEMM_ERR_UNSUPPORTED;
    if (!ld_ok(ldp, 2 * I) || !ld_ok(lddp, 2 * I) || !ld_ok(lddh, I)) return GEMM_ERR_INVALID_VALUE;
    if (ldp > kMaxLd || lddp > kMaxLd || lddh > kMaxLd) return GEMM_ERR_UNSUPPORTED;
    if (rows == 0 || I == 0) return GEMM_OK;
    if (pre == nullptr || dh == nullptr || dpre == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (!aligned(pre, 2) || !aligned(dpre, 2) || !aligned(dh, size_of(dh_type))) return GEMM_ERR_MISALIGNED;
    DeviceInfo dev;
    const gemm_status_t s = usable(dev);
    if (s != GEMM_OK) return s;
    return from_cuda(launch_gated_silu_backward(type, dh_type, rows, I, pre, ldp, dh, lddh, dpre, lddp,
                                                static_cast<cudaStream_t>(stream)));
}

// Rules of the matrices that TMA and 16-byte accesses read and write.
static bool tiled(const void *p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

gemm_status_t gemm_grouped_linear(gemm_type_t type, gemm_type_t y_type, int64_t groups, const int32_t *offsets,
                                  gemm_op_t opW, int gated, int64_t N, int64_t K, const void *X, int64_t ldx,
                                  int64_t x_rows, const int32_t *rows, const void *W, int64_t ldw, int64_t strideW,
                                  void *Y, int64_t ldy, int64_t y_rows, void *pre, int64_t ldp, void *work,
                                  void *stream)
{
    if (!is_type16(type) || (y_type != type && y_type != GEMM_TYPE_F32) || (opW != GEMM_OP_N && opW != GEMM_OP_T) ||
        (gated && opW != GEMM_OP_T) || (!gated && pre != nullptr) || groups < 0 || N < 0 || K < 0 || x_rows < 0 ||
        y_rows < 0 || strideW < 0)
        return GEMM_ERR_INVALID_VALUE;
    if (groups > 1024 || N > kMaxDim24 || K > kMaxDim24 || x_rows > kMaxInt || y_rows > kMaxInt || strideW > kMaxStride)
        return GEMM_ERR_UNSUPPORTED;
    const int64_t w_rows = opW == GEMM_OP_T ? (gated ? 2 * N : N) : K, w_cols = opW == GEMM_OP_T ? K : N;
    if (!ld_ok(ldx, K) || !ld_ok(ldw, w_cols) || !ld_ok(ldy, N) || (pre != nullptr && !ld_ok(ldp, 2 * N)))
        return GEMM_ERR_INVALID_VALUE;
    if (ldx > kMaxLd || ldw > kMaxLd || ldy > kMaxLd || ldp > kMaxLd) return GEMM_ERR_UNSUPPORTED;
    if (groups == 0 || y_rows == 0 || N == 0) return GEMM_OK;
    if (offsets == nullptr || Y == nullptr || (K > 0 && (W == nullptr || (X == nullptr && x_rows > 0))))
        return GEMM_ERR_INVALID_VALUE;
    if (groups > 1 && w_rows > 0 && strideW != 0 && strideW < (w_rows - 1) * ldw + w_cols) return GEMM_ERR_INVALID_VALUE;
    if ((K > 0 && (!tiled(X, ldx) || !tiled(W, ldw) || strideW % 8 != 0)) || !tiled(Y, ldy) ||
        !words(offsets, rows) || (pre != nullptr && !tiled(pre, ldp)) || !aligned(work, 16))
        return GEMM_ERR_MISALIGNED;
    DeviceInfo dev;
    const gemm_status_t s = usable(dev);
    if (s != GEMM_OK) return s;
    const GroupedArgs a{type, y_type, int(groups), offsets, opW, gated != 0, N, K, X, ldx, x_rows, rows, W, ldw, strideW,
                        Y, ldy, y_rows, pre, ldp, Adapters{}, work};
    return launch_grouped(dev, a, static_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_grouped_weight_grad(gemm_type_t type, gemm_type_t dw_type, int64_t groups, const int32_t *offsets,
                                       int64_t N, int64_t K, const void *dY, int64_t lddy, const void *X, int64_t ldx,
                                       int64_t positions, void *dW, int64_t lddw, int64_t strideDW, void *stream)
{
    if (!is_type16(type) || (dw_type != type && dw_type != GEMM_TYPE_F32) || groups < 0 || N < 0 || K < 0 ||
        positions < 0 || strideDW < 0)
        return GEMM_ERR_INVALID_VALUE;
    if (groups > 1024 || N > kMaxDim24 || K > kMaxDim24 || positions > kMaxInt || strideDW > kMaxStride)
        return GEMM_ERR_UNSUPPORTED;
    if (!ld_ok(lddy, N) || !ld_ok(ldx, K) || !ld_ok(lddw, K)) return GEMM_ERR_INVALID_VALUE;
    if (lddy > kMaxLd || ldx > kMaxLd || lddw > kMaxLd) return GEMM_ERR_UNSUPPORTED;
    if (groups == 0 || N == 0 || K == 0) return GEMM_OK;
    if (offsets == nullptr || dW == nullptr || (positions > 0 && (dY == nullptr || X == nullptr)))
        return GEMM_ERR_INVALID_VALUE;
    if (groups > 1 && strideDW < (N - 1) * lddw + K) return GEMM_ERR_INVALID_VALUE;
    if (!tiled(dY, lddy) || !tiled(X, ldx) || !tiled(dW, lddw) || strideDW % 8 != 0 || !words(offsets))
        return GEMM_ERR_MISALIGNED;
    DeviceInfo dev;
    const gemm_status_t s = usable(dev);
    if (s != GEMM_OK) return s;
    const WeightGradArgs a{type, dw_type, int(groups), offsets, N, K, dY, lddy, X, ldx, positions, dW, lddw, strideDW};
    return from_cuda(launch_weight_grad(dev, a, static_cast<cudaStream_t>(stream)));
}

// Partial sums for the device at hand or, without one, for 152 SMs.
static int64_t lora_split_bytes(int64_t T, int64_t N, int64_t K)
{
    DeviceInfo dev;
    return (split_bytes(T, N, K, current_device(dev) ? dev.num_sms / 2 : 76) + 15) / 16 * 16;
}
static int64_t lora_inner_bytes(int64_t T, int64_t requests, int64_t R)
{
    const int64_t few = 4 * T * (R + 1), many = inner_layout(T, requests, R, 3).bytes();
    return ((few > many ? few : many) + 15) / 16 * 16;
}

int64_t gemm_lora_work_bytes(int64_t T, int64_t N, int64_t K, int64_t requests, int64_t R)
{
    if (T <= 0 || N <= 0 || K <= 0 || requests <= 0 || R <= 0 || T > kMaxDim24 || N > kMaxDim24 || K > kMaxDim24 ||
        requests > kMaxDim24 || R > 128)
        return 0;
    return lora_inner_bytes(T, requests, R) + lora_split_bytes(T, N, K);
}

gemm_status_t gemm_lora_linear(gemm_type_t type, gemm_type_t y_type, int64_t T, int64_t N, int64_t K, const void *X,
                               int64_t ldx, const void *W, int64_t ldw, int64_t requests, const int32_t *segments,
                               const int32_t *adapters, int64_t n_adapters, int64_t R, const void *A, int64_t lda,
                               int64_t strideA, const void *B, int64_t ldb, int64_t strideB, const float *scales, void *Y,
                               int64_t ldy, void *work, void *stream)
{
    if (!is_type16(type) || (y_type != type && y_type != GEMM_TYPE_F32) || T < 0 || N < 0 || K < 0 || requests < 0 ||
        n_adapters < 0 || R < 0 || strideA < 0 || strideB < 0)
        return GEMM_ERR_INVALID_VALUE;
    if (T > kMaxDim24 || N > kMaxDim24 || K > kMaxDim24 || requests > kMaxDim24 || n_adapters > kMaxInt || R > 128 ||
        strideA > kMaxStride || strideB > kMaxStride)
        return GEMM_ERR_UNSUPPORTED;
    if (requests > 0 && (T / 32 + requests) * 32 * 6 > kMaxInt) return GEMM_ERR_UNSUPPORTED;
    const bool adapted = requests > 0 && n_adapters > 0 && R > 0 && K > 0;
    if (!ld_ok(ldx, K) || !ld_ok(ldw, K) || !ld_ok(ldy, N) || (adapted && (!ld_ok(lda, K) || !ld_ok(ldb, R))))
        return GEMM_ERR_INVALID_VALUE;
    if (ldx > kMaxLd || ldw > kMaxLd || ldy > kMaxLd || lda > kMaxLd || ldb > kMaxLd) return GEMM_ERR_UNSUPPORTED;
    if (T == 0 || N == 0) return GEMM_OK;
    if (Y == nullptr || (K > 0 && (X == nullptr || W == nullptr))) return GEMM_ERR_INVALID_VALUE;
    if ((K > 0 && (!tiled(X, ldx) || !tiled(W, ldw))) || !tiled(Y, ldy)) return GEMM_ERR_MISALIGNED;
    if (adapted) {
        if (segments == nullptr || adapters == nullptr || A == nullptr || B == nullptr || work == nullptr)
            return GEMM_ERR_INVALID_VALUE;
        if (!tiled(A, lda) || !tiled(B, ldb) || strideA % 8 != 0 || strideB % 8 != 0 ||
            !words(segments, adapters, scales) || !aligned(work, 16))
            return GEMM_ERR_MISALIGNED;
    }
    DeviceInfo dev;
    const gemm_status_t s = usable(dev);
    if (s != GEMM_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    GroupedArgs a{type, y_type, 1, nullptr, GEMM_OP_T, 0, N, K, X, ldx, T, nullptr, W, ldw, 0, Y, ldy, T, nullptr, 0,
                  Adapters{}, nullptr};
    if (adapted) {
        const bool few = takes_few_rows(dev, a);
        const int parts = inner_parts(type, y_type);
        int32_t *which = static_cast<int32_t *>(work) + T * R;
        const ShrinkArgs sh{type, T, K, X, ldx, int(requests), segments, adapters, int(n_adapters), int(R), A, lda, strideA,
                            scales, few ? static_cast<float *>(work) : nullptr, which, work, parts};
        const cudaError_t e = launch_shrink(sh, st);
        if (e != cudaSuccess) return from_cuda(e);
        a.ad = Adapters{B, ldb, strideB, int(R), int(n_adapters), work, which, int(requests), parts, segments, adapters};
        a.work = static_cast<char *>(work) + lora_inner_bytes(T, requests, R);
    }
    return launch_grouped(dev, a, st);
}

}  // extern "C"
