// Row movement and elementwise parts of the routed products: rows out to their positions, the
// weighted sum back, its gradient, and the gradient of the gated activation (semantics:
// include/gemm_gb300.h).  All are bound by memory: every row is read and written once in 16-byte
// pieces (8 elements a thread; element by element where a row length or stride is not a multiple of
// 8), sums are fp32, and nothing uses atomics.
#include <cuda_runtime.h>

#include "routed_internal.h"

namespace gemm {
namespace {

constexpr int kThreads = 256;

template <class T, int VEC> __device__ __forceinline__ void get(const T *p, float (&v)[VEC])
{
    if constexpr (VEC == 8) load8<T>(p, v);
    else v[0] = to_f32(p[0]);
}
template <class T, int VEC> __device__ __forceinline__ void put(T *p, const float (&v)[VEC])
{
    if constexpr (VEC == 8) store8<T>(p, v);
    else p[0] = from_f32<T>(v[0]);
}

// Row and column piece of this thread among rows of `cols` pieces; a 32-bit division where the grid
// allows it (the 64-bit one costs as much as the rest of the kernel's instructions).
__device__ __forceinline__ void place(int64_t cols, int64_t &row, int64_t &piece)
{
    if (gridDim.x <= 0xffffffffu / kThreads) {
        const unsigned i = blockIdx.x * kThreads + threadIdx.x, c = unsigned(cols);
        row = i / c;
        piece = i % c;
    } else {
        const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
        row = i / cols;
        piece = i - row * cols;
    }
}

// Thread: VEC columns of one token; the k rows of a token are read by the same threads.  8192 tokens of
// 4 rows x 2048 to bf16: 50 us from fp32 rows (6.1 TB/s), 34 from bf16 rows (5.0).
template <class R, class Y, int VEC>
__global__ void __launch_bounds__(kThreads)
combine_kernel(int64_t T, int64_t cols, int k, const R *rows, int64_t ldr, int64_t positions, const int32_t *where,
               const float *weights, Y *y, int64_t ldy)
{
    chain_wait();
    int64_t t, c;
    place(cols, t, c);
    c *= VEC;
    if (t >= T) return;
    float acc[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) acc[v] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += 4) {  // four rows in flight
        float row[4][VEC], w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            int64_t p = j0 + j < k ? where[t * k + j0 + j] : -1;
            if (p >= positions) p = -1;
            w[j] = p < 0 ? 0.0f : weights != nullptr ? weights[t * k + j0 + j] : 1.0f;
            if (p >= 0) {
                get<R, VEC>(rows + p * ldr + c, row[j]);
            } else {
#pragma unroll
                for (int v = 0; v < VEC; ++v) row[j][v] = 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int v = 0; v < VEC; ++v) acc[v] = fmaf(w[j], row[j][v], acc[v]);
    }
    put<Y, VEC>(y + t * ldy + c, acc);
}

// Thread: VEC columns of a row of the sum of `count` matrices, added in order.
template <class Y, int VEC>
__global__ void __launch_bounds__(kThreads)
sum_kernel(int64_t rows, int64_t cols, int count, const float *part, int64_t ldp, Y *y, int64_t ldy)
{
    chain_wait();
    int64_t r, c;
    place(cols, r, c);
    c *= VEC;
    if (r >= rows) return;
    float acc[VEC];
    get<float, VEC>(part + r * ldp + c, acc);
#pragma unroll 4
    for (int n = 1; n < count; ++n) {
        float v[VEC];
        get<float, VEC>(part + (n * rows + r) * ldp + c, v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[j] += v[j];
    }
    put<Y, VEC>(y + r * ldy + c, acc);
}

// Thread: VEC columns of one token, read once and written to kSpread of its slots' positions:
// out[where] = w * x[token].  8192 tokens x 2048, bf16, 4 slots each: 26.5 us (6.3 TB/s); a warp a slot,
// which reads the token once for each, 44 us.
constexpr int kSpread = 8;
template <class X, int VEC>
__global__ void __launch_bounds__(kThreads)
dispatch_kernel(int64_t T, int64_t cols, int k, const X *x, int64_t ldx, int64_t positions, const int32_t *where,
                const float *weights, X *out, int64_t ldo)
{
    chain_wait();
    int64_t t, c;
    place(cols, t, c);
    c *= VEC;
    if (t >= T) return;
    float v[VEC];
    get<X, VEC>(x + t * ldx + c, v);
    const int j0 = blockIdx.y * kSpread;
    int32_t p[kSpread];
    float w[kSpread];
#pragma unroll
    for (int j = 0; j < kSpread; ++j) {  // the look-ups in flight together
        p[j] = j0 + j < k ? load_now(where + t * k + j0 + j) : -1;
        w[j] = j0 + j < k && weights != nullptr ? load_now(weights + t * k + j0 + j) : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < kSpread; ++j) {
        if (p[j] < 0 || p[j] >= positions) continue;
        float u[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) u[i] = v[i] * w[j];
        put<X, VEC>(out + p[j] * ldo + c, u);
    }
}

// Warp: one slot, since the dot product of x[token] and rows[where] runs over the row;
// out[where] = w * x[token] beside it, rounded to x's type, since the two products that read it take 16-bit
// rows (their gradients' error grows as the layer's does).  8192 tokens of 4 bf16 rows x 2048: 47 us (6.4
// TB/s), of fp32 rows 68 (6.4).
template <class X, class R, int VEC>
__global__ void __launch_bounds__(kThreads)
combine_backward_kernel(int64_t slots, int64_t cols, int k, const X *x, int64_t ldx, const R *rows, int64_t ldr,
                        int64_t positions, const int32_t *where, const float *weights, X *out, int64_t ldo,
                        float *dweights)
{
    chain_wait();
    const int64_t s = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (s >= slots) return;
    int64_t p = where[s];
    if (p >= positions) p = -1;
    float dot = 0.0f;
    if (p >= 0) {
        const float w = weights != nullptr ? weights[s] : 1.0f;
        const X *src = x + (s / k) * ldx;
        X *dst = out + p * ldo;
        const R *row = rows + p * ldr;
#pragma unroll 4
        for (int64_t c = lane; c < cols; c += 32) {
            float v[VEC], r[VEC];
            get<X, VEC>(src + c * VEC, v);
            get<R, VEC>(row + c * VEC, r);
#pragma unroll
            for (int i = 0; i < VEC; ++i) dot = fmaf(v[i], r[i], dot);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] *= w;
            put<X, VEC>(dst + c * VEC, v);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) dweights[s] = dot;
}

// Warp: one position.  out[p] = x[rows[p]], zeros where the row is outside x, for the positions of a
// group.  16-bit elements in 16-byte pieces; the last piece of an odd row length element by element.
__global__ void __launch_bounds__(kThreads)
gather_kernel(const int32_t *offsets, int groups, int64_t positions, const uint16_t *x, int64_t ldx, int64_t x_rows,
              const int32_t *rows, int64_t K, uint16_t *out, int64_t ldo)
{
    chain_wait();
    const int64_t p = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (p >= positions || p >= load_now(offsets + groups)) return;
    const int r = load_now(rows + p);
    const bool there = r >= 0 && r < x_rows;
    const uint16_t *src = x + int64_t(there ? r : 0) * ldx;
    uint16_t *dst = out + p * ldo;
#pragma unroll 4
    for (int64_t c = 8 * lane; c + 8 <= K; c += 256) {
        const uint4 v = there ? load_now(reinterpret_cast<const uint4 *>(src + c)) : make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4 *>(dst + c) = v;
    }
    const int64_t c = (K & ~int64_t(7)) + lane;
    if (c < K) dst[c] = there ? src[c] : uint16_t(0);
}

// Thread: VEC columns of a position: with s = 1 / (1 + e^-gate), dgate = dh up s (1 + gate (1 - s)) and
// dup = dh gate s.  32768 rows of 2 x 1024, bf16: 57 us (5.9 TB/s).
template <class X, class D, int VEC>
__global__ void __launch_bounds__(kThreads)
gated_silu_backward_kernel(int64_t rows, int64_t cols, int64_t I, const X *pre, int64_t ldp, const D *dh, int64_t lddh,
                           X *dpre, int64_t lddp)
{
    chain_wait();
    int64_t r, c;
    place(cols, r, c);
    c *= VEC;
    if (r >= rows) return;
    float g[VEC], u[VEC], d[VEC], dg[VEC], du[VEC];
    // plain loads: dpre may be pre
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        g[v] = 0.0f;
        u[v] = 0.0f;
    }
    if constexpr (VEC == 8) {
        const uint4 a = *reinterpret_cast<const uint4 *>(pre + r * ldp + c);
        const uint4 b = *reinterpret_cast<const uint4 *>(pre + r * ldp + I + c);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            g[v] = to_f32(reinterpret_cast<const X *>(&a)[v]);
            u[v] = to_f32(reinterpret_cast<const X *>(&b)[v]);
        }
    } else {
        g[0] = to_f32(pre[r * ldp + c]);
        u[0] = to_f32(pre[r * ldp + I + c]);
    }
    get<D, VEC>(dh + r * lddh + c, d);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        const float s = sigmoid(g[v]);
        dg[v] = d[v] * u[v] * s * (1.0f + g[v] * (1.0f - s));
        du[v] = d[v] * g[v] * s;
    }
    put<X, VEC>(dpre + r * lddp + c, dg);
    put<X, VEC>(dpre + r * lddp + I + c, du);
}

bool wide(const void *p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0; }

template <class F> cudaError_t by_type16(int type, F f)
{
    return type == GEMM_TYPE_F16 ? f(__half{}) : f(__nv_bfloat16{});
}
template <class F> cudaError_t by_type(int type, F f)
{
    return type == GEMM_TYPE_F32 ? f(float{}) : by_type16(type, f);
}
// Grid of n threads or warps in CTAs of `per`; 2^31 CTAs are more than any memory holds rows for.
bool grid_of(int64_t n, int64_t per, unsigned &blocks)
{
    const int64_t b = (n + per - 1) / per;
    blocks = unsigned(b);
    return b < (int64_t(1) << 31);
}

}  // namespace

cudaError_t launch_combine(int rows_type, int y_type, int64_t T, int64_t H, int top_k, const void *rows, int64_t ldr,
                           int64_t positions, const int32_t *where, const float *weights, void *y, int64_t ldy,
                           cudaStream_t stream)
{
    const bool vec = H % 8 == 0 && wide(rows, ldr) && wide(y, ldy);
    const int64_t cols = vec ? H / 8 : H;
    unsigned blocks;
    if (!grid_of(T * cols, kThreads, blocks)) return cudaErrorInvalidConfiguration;
    return by_type(rows_type, [&](auto r) {
        return by_type(y_type, [&](auto o) {
            using R = decltype(r);
            using Y = decltype(o);
            auto *kernel = vec ? combine_kernel<R, Y, 8> : combine_kernel<R, Y, 1>;
            return launch_chained(kernel, dim3(blocks), kThreads, 0, 1, stream, T, cols, top_k, static_cast<const R *>(rows), ldr, positions, where,
                                                    weights, static_cast<Y *>(y), ldy);
        });
    });
}

cudaError_t launch_dispatch(int type, int rows_type, int64_t T, int64_t H, int top_k, const void *x, int64_t ldx,
                            const void *rows, int64_t ldr, int64_t positions, const int32_t *where,
                            const float *weights, void *out, int64_t ldo, float *dweights, cudaStream_t stream)
{
    const bool vec = H % 8 == 0 && wide(x, ldx) && wide(out, ldo) && (rows == nullptr || wide(rows, ldr));
    const int64_t cols = vec ? H / 8 : H;
    unsigned blocks;
    // dispatch alone: a thread a piece of a token; with the weights' gradient: a warp a slot
    if (dweights == nullptr ? !grid_of(T * cols, kThreads, blocks) : !grid_of(T * top_k, kThreads / 32, blocks))
        return cudaErrorInvalidConfiguration;
    return by_type(type, [&](auto a) {
        using X = decltype(a);
        if (dweights == nullptr) {
            const dim3 grid(blocks, unsigned((top_k + kSpread - 1) / kSpread));
            auto *kernel = vec ? dispatch_kernel<X, 8> : dispatch_kernel<X, 1>;
            return launch_chained(kernel, grid, kThreads, 0, 1, stream, T, cols, top_k, static_cast<const X *>(x), ldx,
                                  positions, where, weights, static_cast<X *>(out), ldo);
        }
        return by_type(rows_type, [&](auto r) {
            using R = decltype(r);
            auto *kernel = vec ? combine_backward_kernel<X, R, 8> : combine_backward_kernel<X, R, 1>;
            return launch_chained(kernel, dim3(blocks), kThreads, 0, 1, stream, T * top_k, cols, top_k, static_cast<const X *>(x), ldx,
                                                    static_cast<const R *>(rows), ldr, positions, where, weights,
                                                    static_cast<X *>(out), ldo, dweights);
        });
    });
}

cudaError_t launch_sum(int y_type, int64_t rows, int64_t cols, int count, const float *part, int64_t ldp, void *y, int64_t ldy,
                       cudaStream_t stream)
{
    const bool vec = cols % 8 == 0;  // both matrices' rows start on 16-byte boundaries
    const int64_t pieces = vec ? cols / 8 : cols;
    unsigned blocks;
    if (!grid_of(rows * pieces, kThreads, blocks)) return cudaErrorInvalidConfiguration;
    return by_type(y_type, [&](auto o) {
        using Y = decltype(o);
        auto *kernel = vec ? sum_kernel<Y, 8> : sum_kernel<Y, 1>;
        return launch_chained(kernel, dim3(blocks), kThreads, 0, 1, stream, rows, pieces, count, part, ldp, static_cast<Y *>(y),
                              ldy);
    });
}

cudaError_t launch_gather(const GroupedArgs &a, void *out, int64_t ldo, cudaStream_t stream)
{
    unsigned blocks;
    if (!grid_of(a.y_rows, kThreads / 32, blocks)) return cudaErrorInvalidConfiguration;
    return launch_chained(gather_kernel, dim3(blocks), kThreads, 0, 1, stream, a.offsets, a.groups, a.y_rows, static_cast<const uint16_t *>(a.X), a.ldx,
                                                   a.x_rows, a.rows, a.K, static_cast<uint16_t *>(out), ldo);
}

cudaError_t launch_gated_silu_backward(int type, int dh_type, int64_t rows, int64_t I, const void *pre, int64_t ldp,
                                       const void *dh, int64_t lddh, void *dpre, int64_t lddp, cudaStream_t stream)
{
    const bool vec = I % 8 == 0 && wide(pre, ldp) && wide(dh, lddh) && wide(dpre, lddp);
    const int64_t cols = vec ? I / 8 : I;
    unsigned blocks;
    if (!grid_of(rows * cols, kThreads, blocks)) return cudaErrorInvalidConfiguration;
    return by_type16(type, [&](auto a) {
        using X = decltype(a);
        auto go = [&](auto d) {
            using D = decltype(d);
            auto *kernel = vec ? gated_silu_backward_kernel<X, D, 8> : gated_silu_backward_kernel<X, D, 1>;
            return launch_chained(kernel, dim3(blocks), kThreads, 0, 1, stream, rows, cols, I, static_cast<const X *>(pre), ldp,
                                                    static_cast<const D *>(dh), lddh, static_cast<X *>(dpre), lddp);
        };
        return dh_type == GEMM_TYPE_F32 ? go(float{}) : go(X{});
    });
}

}  // namespace gemm
