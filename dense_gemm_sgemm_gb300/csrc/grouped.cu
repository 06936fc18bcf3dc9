// Grouped products: which kernel takes which call, and the tiled fp32 kernel for the forms without
// a tensor-core kernel.
#include <cuda_runtime.h>

#include "routed_internal.h"

namespace gemm {
namespace {

constexpr int kTile = 64, kStep = 16;

__device__ __forceinline__ int clamp_to(int v, int64_t hi) { return v < 0 ? 0 : v > hi ? int(hi) : v; }

// Y[p] = X[r(p)] W_g with W_g stored K x N: 64 x 64 tiles, 4 x 4 outputs a thread, fp32 multiply-adds.
template <class T, class Y> __global__ void __launch_bounds__(256) grouped_n_kernel(const GroupedArgs a)
{
    __shared__ float xs[kStep][kTile + 4], ws[kStep][kTile + 4];
    const int g = blockIdx.y;
    const int lo = clamp_to(a.offsets[g], a.y_rows), hi = clamp_to(a.offsets[g + 1], a.y_rows);
    const T *W = static_cast<const T *>(a.W) + int64_t(g) * a.stridew;
    const T *X = static_cast<const T *>(a.X);
    const int64_t n0 = int64_t(blockIdx.x) * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    for (int p0 = lo + int(blockIdx.z) * kTile; p0 < hi; p0 += int(gridDim.z) * kTile) {
        float acc[4][4] = {};
        for (int64_t k0 = 0; k0 < a.K; k0 += kStep) {
            for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
                const int k = i % kStep, p = p0 + i / kStep;
                int64_t r = p < hi ? (a.rows != nullptr ? a.rows[p] : p) : -1;
                if (r >= a.x_rows) r = -1;
                xs[k][i / kStep] = r >= 0 && k0 + k < a.K ? to_f32(X[r * a.ldx + k0 + k]) : 0.0f;
                const int n = i % kTile, kk = i / kTile;
                ws[kk][n] = n0 + n < a.N && k0 + kk < a.K ? to_f32(W[(k0 + kk) * a.ldw + n0 + n]) : 0.0f;
            }
            __syncthreads();
            for (int k = 0; k < kStep; ++k)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[k][4 * ty + i], ws[k][4 * tx + j], acc[i][j]);
            __syncthreads();
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int p = p0 + 4 * ty + i;
                const int64_t n = n0 + 4 * tx + j;
                if (p < hi && n < a.N) static_cast<Y *>(a.Y)[p * a.ldy + n] = from_f32<Y>(acc[i][j]);
            }
    }
}

template <class T, class Y> __global__ void __launch_bounds__(256) weight_grad_kernel(const WeightGradArgs a)
{
    __shared__ float ds[kStep][kTile + 4], xs[kStep][kTile + 4];
    const int g = blockIdx.z;
    const int lo = clamp_to(a.offsets[g], a.positions), hi = clamp_to(a.offsets[g + 1], a.positions);
    const int64_t n0 = int64_t(blockIdx.y) * kTile, k0 = int64_t(blockIdx.x) * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int p0 = lo; p0 < hi; p0 += kStep) {
        for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
            const int c = i % kTile, r = i / kTile;
            const int64_t p = p0 + r;
            ds[r][c] = p < hi && n0 + c < a.N ? to_f32(static_cast<const T *>(a.dY)[p * a.lddy + n0 + c]) : 0.0f;
            xs[r][c] = p < hi && k0 + c < a.K ? to_f32(static_cast<const T *>(a.X)[p * a.ldx + k0 + c]) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < kStep; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(ds[k][4 * ty + i], xs[k][4 * tx + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + 4 * ty + i, k = k0 + 4 * tx + j;
            if (n < a.N && k < a.K)
                static_cast<Y *>(a.dW)[int64_t(g) * a.stridedw + n * a.lddw + k] = from_f32<Y>(acc[i][j]);
        }
}

cudaError_t counted()
{
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches();
    return e;
}

template <class F> cudaError_t by_types(int type, int out_type, F f)
{
    if (type == GEMM_TYPE_F16) return out_type == GEMM_TYPE_F32 ? f(__half{}, float{}) : f(__half{}, __half{});
    return out_type == GEMM_TYPE_F32 ? f(__nv_bfloat16{}, float{}) : f(__nv_bfloat16{}, __nv_bfloat16{});
}

}  // namespace

gemm_status_t launch_grouped(const DeviceInfo &dev, const GroupedArgs &a, cudaStream_t stream)
{
    if (a.opW == GEMM_OP_T) return launch_few_rows(dev, a, stream) == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
    const cudaError_t e = by_types(a.type, a.y_type, [&](auto t, auto y) {
        const dim3 grid(unsigned((a.N + kTile - 1) / kTile), unsigned(a.groups),
                        unsigned(a.y_rows / a.groups / kTile + 1 < 64 ? a.y_rows / a.groups / kTile + 1 : 64));
        grouped_n_kernel<decltype(t), decltype(y)><<<grid, 256, 0, stream>>>(a);
        return counted();
    });
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

gemm_status_t launch_weight_grad(const DeviceInfo &, const WeightGradArgs &a, cudaStream_t stream)
{
    const cudaError_t e = by_types(a.type, a.dw_type, [&](auto t, auto y) {
        const dim3 grid(unsigned((a.K + kTile - 1) / kTile), unsigned((a.N + kTile - 1) / kTile), unsigned(a.groups));
        weight_grad_kernel<decltype(t), decltype(y)><<<grid, 256, 0, stream>>>(a);
        return counted();
    });
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace gemm
