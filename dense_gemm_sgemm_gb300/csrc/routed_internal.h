// Declarations shared by the routed products: routing, row movement, grouped products and
// adapters.  The launchers take validated arguments (routed_api.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gemm_internal.h"

namespace gemm {

// 16-bit storage types and their conversions; everything is computed in fp32.
template <class T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }

// Eight consecutive elements, 16-byte aligned.
template <class T> __device__ __forceinline__ void load8(const T *p, float (&v)[8])
{
    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
    const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
}
template <> __device__ __forceinline__ void load8(const float *p, float (&v)[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <class T> __device__ __forceinline__ void store8(T *p, const float (&v)[8])
{
    uint4 u;
    T *e = reinterpret_cast<T *>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(v[i]);
    *reinterpret_cast<uint4 *>(p) = u;
}
template <> __device__ __forceinline__ void store8(float *p, const float (&v)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// 1 / (1 + exp(-x)); 0 and 1 at the ends, no NaN for finite x.
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Lets `kernel` use up to `bytes` of dynamic shared memory; asks the runtime once per kernel and
// device (the call costs as much as a launch), so every call of one kernel names the same bytes.
cudaError_t allow_smem_once(const void *kernel, int bytes);
template <class... P> cudaError_t allow_smem_once(void (*kernel)(P...), int bytes)
{
    return allow_smem_once(reinterpret_cast<const void *>(kernel), bytes);
}

// Likewise lets `kernel` run in clusters of more than the portable 8 CTAs.
cudaError_t allow_large_cluster_once(const void *kernel);
template <class... P> cudaError_t allow_large_cluster_once(void (*kernel)(P...))
{
    return allow_large_cluster_once(reinterpret_cast<const void *>(kernel));
}

struct RouteArgs {
    int type;
    int64_t T;
    int E;
    const void *logits;
    int64_t ld;
    const float *bias;
    int score, groups, groups_kept, group_top, top_k, renormalise;
    float scale;
    int32_t *ids;
    float *weights;
    int32_t *offsets, *tokens, *where;
    bool wide;  // set by the launcher: rows of logits start on 16-byte boundaries
};
cudaError_t launch_route(const RouteArgs &a, cudaStream_t stream);
cudaError_t launch_plan(int64_t T, int E, int top_k, const int32_t *ids, int32_t *offsets, int32_t *tokens,
                        int32_t *where, cudaStream_t stream);
cudaError_t launch_route_backward(const RouteArgs &a, const float *dweights, const int32_t *ids, void *dlogits,
                                  int64_t ldd, cudaStream_t stream);

cudaError_t launch_combine(int rows_type, int y_type, int64_t T, int64_t H, int top_k, const void *rows, int64_t ldr,
                           int64_t positions, const int32_t *where, const float *weights, void *y, int64_t ldy,
                           cudaStream_t stream);
// out[where] = w * x, and with dweights the dot products of x and rows (gemm_moe_combine_backward).
cudaError_t launch_dispatch(int type, int rows_type, int64_t T, int64_t H, int top_k, const void *x, int64_t ldx,
                            const void *rows, int64_t ldr, int64_t positions, const int32_t *where,
                            const float *weights, void *out, int64_t ldo, float *dweights, cudaStream_t stream);
cudaError_t launch_gated_silu_backward(int type, int dh_type, int64_t rows, int64_t I, const void *pre, int64_t ldp,
                                       const void *dh, int64_t lddh, void *dpre, int64_t lddp, cudaStream_t stream);

// A product of a grouped linear layer or of a linear layer with adapters: positions are split into
// groups by offsets (NULL: one group of all y_rows positions), every group has its own W.
struct Adapters {
    const void *b;         // NULL: no adapters
    int64_t ldb, strideb;
    int rank, count;
    const float *inner;    // y_rows x rank: scale * X A^T of each position's adapter
    const int32_t *which;  // y_rows: adapter of each position, -1: none
};
struct GroupedArgs {
    int type, y_type;
    int groups;
    const int32_t *offsets;
    int opW, gated;
    int64_t N, K;
    const void *X;
    int64_t ldx, x_rows;
    const int32_t *rows;
    const void *W;
    int64_t ldw, stridew;
    void *Y;
    int64_t ldy, y_rows;
    void *pre;
    int64_t ldp;
    Adapters ad;
    void *work;  // y_rows x (K rounded up to 8) elements, or NULL
};
// Few rows per group (opW = T): weights straight from global memory to mma.sync fragments.
cudaError_t launch_few_rows(const DeviceInfo &dev, const GroupedArgs &a, cudaStream_t stream);

// Many rows per group, or opW = N: tcgen05 tiles fed by TMA.
cudaError_t launch_many_rows(const DeviceInfo &dev, const GroupedArgs &a, cudaStream_t stream);
// X[rows[p]] to row p of `out`, for the positions of the groups.
cudaError_t launch_gather(const GroupedArgs &a, void *out, int64_t ldo, cudaStream_t stream);
gemm_status_t launch_grouped(const DeviceInfo &dev, const GroupedArgs &a, cudaStream_t stream);

struct WeightGradArgs {
    int type, dw_type;
    int groups;
    const int32_t *offsets;
    int64_t N, K;
    const void *dY;
    int64_t lddy;
    const void *X;
    int64_t ldx, positions;
    void *dW;
    int64_t lddw, stridedw;
};
cudaError_t launch_weight_grad(const DeviceInfo &dev, const WeightGradArgs &a, cudaStream_t stream);

struct ShrinkArgs {
    int type;
    int64_t T, K;
    const void *X;
    int64_t ldx;
    int requests;
    const int32_t *segments, *adapters;
    int n_adapters, R;
    const void *A;
    int64_t lda, stridea;
    const float *scales;
    float *inner;
    int32_t *which;
};
cudaError_t launch_shrink(const ShrinkArgs &a, cudaStream_t stream);

}  // namespace gemm
