// Declarations shared by the routed products: routing, row movement, grouped products and
// adapters.  The launchers take validated arguments (routed_api.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "gemm_internal.h"

namespace gemm {

// The routed products' kernels follow one another closely: each is launched so that it may take its
// place on the SMs before the kernel ahead of it on the stream has ended, and begins with
// chain_wait(), which returns once that kernel has ended and its writes are visible, and which lets
// the next kernel take its place in turn.  Before it a kernel may only set up its own SM.
__device__ __forceinline__ void chain_wait()
{
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}
template <class K, class... Args>
cudaError_t launch_chained(K *kernel, dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream, const Args &...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e == cudaSuccess) count_launches();
    return e;
}

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

// Elements [k, k + 8) of a 16-bit row of K elements, 16-byte aligned: zeros beyond K, nothing read there.
template <class T> __device__ __forceinline__ uint4 load_tail(const T *row, int64_t k, int64_t K)
{
    if (k + 8 <= K) return __ldg(reinterpret_cast<const uint4 *>(row + k));
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    const uint16_t *src = reinterpret_cast<const uint16_t *>(row);
    uint16_t *dst = reinterpret_cast<uint16_t *>(&v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < K) dst[i] = __ldg(src + k + i);
    return v;
}

// c += A B with mma.sync m16n8k16, fp32 accumulation.  Lane (g, t) = (lane / 4, lane % 4) holds two
// k each of A's rows g (a0, a2) and g + 8 (a1, a3), of B's column g (b0, b1), and of c the columns
// 2 t, 2 t + 1 of rows g and g + 8.
template <class T>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    if constexpr (std::is_same<T, __half>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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
// The products scale * X A^T of each token with its adapter reach the second product in one of two
// forms.  For the few-rows kernel: fp32, a row of `rank` for every token, and its adapter in `which`.
// For the tcgen05 kernel: 16-bit parts that sum to the fp32 value, part i of 64 ranks in plane i *
// blocks + block, rows of 64; tokens in blocks of 32, where block b of request q is rows 32 (b + q) ..
// of a plane and tokens of other requests are zeros, so that one request's blocks are contiguous.
// Behind the planes the fp32 values, as the few-rows kernel takes them: where a part or a zero does not
// stand for its value (0 * inf) the tcgen05 kernel's epilogue takes them too (TileRequests).
struct InnerLayout {
    int parts, blocks;
    int64_t plane_rows, values;
    __host__ __device__ int64_t values_at() const { return plane_rows * 128 * parts * blocks; }
    __host__ __device__ int64_t bytes() const { return values_at() + 4 * values; }
};
// Parts: fp16's two hold 22 bits from 2^-3 up and the multiples of 2^-24 below it, an error of 2^-25 at
// most: next to the products that they are added to that matters to values of that size only, and a third
// part would have the same spacing.  bf16's two hold 16, 2^8 times finer than a 16-bit output; an fp32
// output takes three.
inline int inner_parts(int type, int y_type) { return type == GEMM_TYPE_BF16 && y_type == GEMM_TYPE_F32 ? 3 : 2; }
__host__ __device__ inline InnerLayout inner_layout(int64_t tokens, int64_t requests, int64_t rank, int parts)
{
    return InnerLayout{parts, int((rank + 63) / 64), (tokens / 32 + requests) * 32, tokens * rank};
}
struct Adapters {
    const void *b;  // NULL: no adapters
    int64_t ldb, strideb;
    int rank, count;
    const void *inner;
    const int32_t *which;  // few-rows kernel: adapter of each position, -1: none
    int requests, parts;   // tcgen05 kernel
    const int32_t *segments, *adapters;
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
    // gathered rows: y_rows x (K rounded up to 64) elements; adapters: split_bytes() of partial sums; or
    // NULL
    void *work;
};
// Bytes of the partial sums of a linear layer with adapters on a device of 2 * pairs SMs.
int64_t split_bytes(int64_t rows, int64_t N, int64_t K, int pairs);
// y = the sum of `count` fp32 matrices of rows x cols, rows * ldp elements apart.
cudaError_t launch_sum(int y_type, int64_t rows, int64_t cols, int count, const float *part, int64_t ldp, void *y, int64_t ldy,
                       cudaStream_t stream);
// Few rows per group (opW = T): weights straight from global memory to mma.sync fragments.
cudaError_t launch_few_rows(const DeviceInfo &dev, const GroupedArgs &a, cudaStream_t stream);

// Many rows per group, or opW = N: tcgen05 tiles fed by TMA.
cudaError_t launch_many_rows(const DeviceInfo &dev, const GroupedArgs &a, cudaStream_t stream);
// X[rows[p]] to row p of `out`, for the positions of the groups.
cudaError_t launch_gather(const GroupedArgs &a, void *out, int64_t ldo, cudaStream_t stream);
bool takes_few_rows(const DeviceInfo &dev, const GroupedArgs &a);
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
    float *inner;    // few-rows form, NULL: the other
    int32_t *which;
    void *planes;    // tcgen05 form, of `parts`, and the fp32 values
    int n_parts;
};
cudaError_t launch_shrink(const ShrinkArgs &a, cudaStream_t stream);

}  // namespace gemm
