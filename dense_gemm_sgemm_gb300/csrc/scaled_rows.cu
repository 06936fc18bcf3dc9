// Block-scaled 8-bit values: quantising in blocks of 1 x 128, 128 x 1 or 128 x 128 elements, and reading
// back (semantics: include/gemm_gb300.h).
//
// A block's scale is a power of two, so x / s only moves the exponent and an element is rounded once, to
// its 8-bit value: any arithmetic gives the same codes, and a value quantised along rows and along columns
// is off by its own rounding alone.  Powers of two cost up to one bit of the 8-bit types' range (not of
// their precision).
//
// Bound by memory: every element is read once, written once per way of quantising.  A CTA holds a tile of
// 128 x 128 elements in registers (64 a thread), from which the maxima along rows (shuffles), along
// columns and of the tile (shared memory) all follow in the one pass.
#include <cuda_runtime.h>

#include <cfloat>

#include "scaled_internal.h"

namespace gemm {
namespace {

constexpr int kThreads = 256;
constexpr unsigned kFull = 0xffffffffu;
constexpr int kRows = 1, kColumns = 2, kTiles = 4;

// |x| for the maximum of a block; infinities and NaN take no part.
__device__ __forceinline__ float magnitude(float x)
{
    const float a = fabsf(x);
    return a <= FLT_MAX ? a : 0.0f;
}

// The power of two with max <= s * 1.75 * 2^top, top the exponent of the type's largest value 1.75 * 2^top:
// its biased exponent, at least 1 (2^-126); 127 (a scale of 1) for a block of zeros.
__device__ __forceinline__ uint32_t scale_exponent(float max, int top)
{
    if (max == 0.0f) return 127u;
    const uint32_t u = __float_as_uint(max);
    const int e = int(u >> 23) - top + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return uint32_t(e < 1 ? 1 : e);
}
__device__ __forceinline__ float power(uint32_t exponent) { return __uint_as_float(exponent << 23); }

// Eight values times the reciprocal scale 2^(127 - exponent) as 8-bit codes.  An infinity is stored as NaN
// like NaN itself: neither turns finite, e4m3 has no infinity.
__device__ __forceinline__ uint2 codes(const float (&v)[8], const uint32_t (&exponent)[8], bool e5m2)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f;
        f.x = v[2 * i] * power(254u - exponent[2 * i]);
        f.y = v[2 * i + 1] * power(254u - exponent[2 * i + 1]);
        if (!(fabsf(f.x) <= FLT_MAX)) f.x = __uint_as_float(0x7fffffffu);
        if (!(fabsf(f.y) <= FLT_MAX)) f.y = __uint_as_float(0x7fffffffu);
        w[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, e5m2 ? __NV_E5M2 : __NV_E4M3);
    }
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

__device__ __forceinline__ void put_codes(uint8_t *q, uint2 w, int64_t left)
{
    if (left >= 8) {
        *reinterpret_cast<uint2 *>(q) = w;
    } else {
        const uint64_t u = uint64_t(w.y) << 32 | w.x;
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < left) q[i] = uint8_t(u >> (8 * i));
    }
}

struct QuantizeParams {
    int64_t rows, cols, ldx, ldq, ldqc;
    const void *X;
    uint8_t *Q, *Qc;
    Scales s, sc;
    int col_blocks, wide, e5m2;
};

// Thread (x, y) = (t % 16, t / 16): 8 columns of the rows y, y + 16, .. of a tile of 16 * I rows.  MODE: the
// sum of the ways.  Blocks of 1 x 128 alone do not need a tile's height: few rows take I = 1, for more CTAs.
template <class T, int MODE, int I>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantizeParams p)
{
    __shared__ float column_max[MODE & kColumns ? 16 : 1][128];
    __shared__ uint32_t column_exponent[128];
    __shared__ float warp_max[kThreads / 32];
    chain_wait();
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4, top = p.e5m2 ? 15 : 8;
    const int64_t rb = blockIdx.x / unsigned(p.col_blocks), cb = blockIdx.x % unsigned(p.col_blocks);
    const int64_t r0 = rb * (16 * I) + y, c = cb * 128 + x * 8, left = p.cols - c;
    const T *src = static_cast<const T *>(p.X) + r0 * p.ldx + c;
    float v[I][8];
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const bool in = r0 + 16 * i < p.rows;
        if (in && p.wide && left >= 8) {
            load8<T>(src + int64_t(16 * i) * p.ldx, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = in && j < left ? to_f32(src[int64_t(16 * i) * p.ldx + j]) : 0.0f;
        }
    }
    if constexpr ((MODE & kRows) != 0) {
#pragma unroll
        for (int i = 0; i < I; ++i) {
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, magnitude(v[i][j]));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
            const uint32_t e = scale_exponent(m, top);
            const uint32_t all[8] = {e, e, e, e, e, e, e, e};
            const int64_t r = r0 + 16 * i;
            if (r >= p.rows) continue;
            if (x == 0) p.s.at[r * p.s.row + cb * p.s.col] = power(e);
            if (left > 0) put_codes(p.Q + r * p.ldq + c, codes(v[i], all, p.e5m2), left);
        }
    }
    if constexpr ((MODE & kTiles) != 0) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, magnitude(v[i][j]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
        __syncthreads();
        m = warp_max[0];
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) m = fmaxf(m, warp_max[i]);
        const uint32_t e = scale_exponent(m, top);
        const uint32_t all[8] = {e, e, e, e, e, e, e, e};
        if (threadIdx.x == 0) p.s.at[rb * p.s.row + cb * p.s.col] = power(e);
#pragma unroll
        for (int i = 0; i < I; ++i)
            if (r0 + 16 * i < p.rows && left > 0)
                put_codes(p.Q + (r0 + 16 * i) * p.ldq + c, codes(v[i], all, p.e5m2), left);
    }
    if constexpr ((MODE & kColumns) != 0) {
        float m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < I; ++i) m[j] = fmaxf(m[j], magnitude(v[i][j]));
        }
        float4 *to = reinterpret_cast<float4 *>(&column_max[y][x * 8]);
        to[0] = make_float4(m[0], m[1], m[2], m[3]);
        to[1] = make_float4(m[4], m[5], m[6], m[7]);
        __syncthreads();
        if (threadIdx.x < 128) {
            float most = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) most = fmaxf(most, column_max[i][threadIdx.x]);
            const uint32_t e = scale_exponent(most, top);
            column_exponent[threadIdx.x] = e;
            const int64_t col = cb * 128 + threadIdx.x;
            if (col < p.cols) p.sc.at[rb * p.sc.row + col * p.sc.col] = power(e);
        }
        __syncthreads();
        uint32_t e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = column_exponent[x * 8 + j];
#pragma unroll
        for (int i = 0; i < I; ++i)
            if (r0 + 16 * i < p.rows && left > 0)
                put_codes(p.Qc + (r0 + 16 * i) * p.ldqc + c, codes(v[i], e, p.e5m2), left);
    }
}

template <class T> cudaError_t quantize(const QuantizeArgs &a, cudaStream_t stream)
{
    QuantizeParams p{};
    p.rows = a.rows;
    p.cols = a.cols;
    p.X = a.X;
    p.ldx = a.ldx;
    p.Q = static_cast<uint8_t *>(a.Q);
    p.ldq = a.ldq;
    p.s = a.s;
    p.Qc = static_cast<uint8_t *>(a.Qc);
    p.ldqc = a.ldqc;
    p.sc = a.sc;
    p.e5m2 = a.q_type == GEMM_TYPE_E5M2;
    p.wide = reinterpret_cast<uintptr_t>(a.X) % 16 == 0 && a.ldx * int64_t(sizeof(T)) % 16 == 0;
    const int64_t blocks = (a.cols + 127) / 128;
    p.col_blocks = int(blocks);
    const bool rows_alone = a.Qc == nullptr && a.s.row_shift == 0;
    // few rows: 16 a CTA (64 x 4096 on 128 CTAs instead of 32)
    const bool few = rows_alone && ((a.rows + 127) / 128) * blocks < 304;
    const int64_t height = few ? 16 : 128, grid = (a.rows + height - 1) / height * blocks;
    if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    const dim3 g{unsigned(grid)};
    if (few) return launch_chained(quantize_kernel<T, kRows, 1>, g, kThreads, 0, 1, stream, p);
    if (rows_alone) return launch_chained(quantize_kernel<T, kRows, 8>, g, kThreads, 0, 1, stream, p);
    if (a.Q == nullptr) return launch_chained(quantize_kernel<T, kColumns, 8>, g, kThreads, 0, 1, stream, p);
    if (a.Qc == nullptr) return launch_chained(quantize_kernel<T, kTiles, 8>, g, kThreads, 0, 1, stream, p);
    return launch_chained(quantize_kernel<T, kRows + kColumns, 8>, g, kThreads, 0, 1, stream, p);
}

// Thread: 16 columns of one row.  A 128-wide block's scale serves all of them.
template <class Y>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(int64_t rows, int64_t cols, const uint8_t *Q, int64_t ldq, const Scales s, Y *y, int64_t ldy,
                  int wide, int e5m2)
{
    chain_wait();
    const int64_t r = int64_t(blockIdx.x) * (kThreads / 16) + (threadIdx.x >> 4);
    if (r >= rows) return;
    const float *at = s.at + (r >> s.row_shift) * s.row;
    for (int64_t c = (int64_t(blockIdx.y) * 16 + (threadIdx.x & 15)) * 16; c < cols; c += int64_t(gridDim.y) * 256) {
        const int64_t left = cols - c;
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (left >= 16) {
            const uint4 u = __ldg(reinterpret_cast<const uint4 *>(Q + r * ldq + c));
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else {
            for (int i = 0; i < left; ++i) w[i / 4] |= uint32_t(Q[r * ldq + c + i]) << (8 * (i & 3));
        }
        float f[2][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t two = uint16_t(w[i / 2] >> (16 * (i & 1)));
            const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(two, e5m2 ? __NV_E5M2 : __NV_E4M3));
            const float2 v = __half22float2(h);
            f[i / 4][2 * (i % 4)] = v.x;
            f[i / 4][2 * (i % 4) + 1] = v.y;
        }
        if (s.col_shift != 0) {
            const float m = __ldg(at + (c >> s.col_shift) * s.col);
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i / 8][i % 8] *= m;
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < left) f[i / 8][i % 8] *= __ldg(at + (c + i) * s.col);
        }
        Y *to = y + r * ldy + c;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (wide && left >= 8 * (h + 1)) {
                store8<Y>(to + 8 * h, f[h]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (8 * h + i < left) to[8 * h + i] = from_f32<Y>(f[h][i]);
            }
        }
    }
}

template <class Y>
cudaError_t dequantize(int q_type, int64_t rows, int64_t cols, const void *Q, int64_t ldq, const Scales &s, void *y, int64_t ldy,
                       cudaStream_t stream)
{
    const int wide = reinterpret_cast<uintptr_t>(y) % 16 == 0 && ldy * int64_t(sizeof(Y)) % 16 == 0;
    const int64_t tall = (rows + 15) / 16, across = (cols + 255) / 256;
    if (tall >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    const dim3 grid(unsigned(tall), unsigned(across < 65535 ? across : 65535));
    return launch_chained(dequantize_kernel<Y>, grid, kThreads, 0, 1, stream, rows, cols, static_cast<const uint8_t *>(Q), ldq, s,
                          static_cast<Y *>(y), ldy, wide, int(q_type == GEMM_TYPE_E5M2));
}

}  // namespace

cudaError_t launch_quantize(const QuantizeArgs &a, cudaStream_t stream)
{
    if (a.type == GEMM_TYPE_F32) return quantize<float>(a, stream);
    if (a.type == GEMM_TYPE_F16) return quantize<__half>(a, stream);
    return quantize<__nv_bfloat16>(a, stream);
}

cudaError_t launch_dequantize(int q_type, int y_type, int64_t rows, int64_t cols, const void *Q, int64_t ldq, const Scales &s, void *Y,
                              int64_t ldy, cudaStream_t stream)
{
    if (y_type == GEMM_TYPE_F32) return dequantize<float>(q_type, rows, cols, Q, ldq, s, Y, ldy, stream);
    if (y_type == GEMM_TYPE_F16) return dequantize<__half>(q_type, rows, cols, Q, ldq, s, Y, ldy, stream);
    return dequantize<__nv_bfloat16>(q_type, rows, cols, Q, ldq, s, Y, ldy, stream);
}

}  // namespace gemm
