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
// columns and of the tile (shared memory) all follow in the one pass.  16384 x 4096 (GB300, copies 6.77 TB/s): bf16
// by rows 32 us (6.4 TB/s), 128 x 128 32 (6.3), columns 33 (6.1), rows and columns 43 (6.3); fp32 50, 50, 51 and 62
// (6.5 to 6.7); read back to bf16 32 (6.3), to fp32 51 (6.6).  64 x 4096 by rows: 1.8 us, a launch and one chain of
// latencies.  For 16-bit types three CTAs an SM have to fit (two: 35 to 50 us), hence the maxima in pairs, the
// conversions repeated rather than kept, and the column maxima handed over before the rows.  Rows that do not begin
// on 16-byte boundaries are read element by element (4095 x 4097: 14.5 to 26 us in bf16; through the aligned
// pieces around them, shifted, it was no faster and fp32 a third slower).
#include <cuda_runtime.h>

#include <cfloat>

#include "scaled_internal.h"

namespace gemm {
namespace {

constexpr int kThreads = 256;
constexpr unsigned kFull = 0xffffffffu;
constexpr int kRows = 1, kColumns = 2, kTiles = 4;

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

// Eight consecutive elements of a row as they are in memory (16-bit types take half the registers of floats),
// and as floats.  left: elements before the row's end.
template <class T> struct Piece {
    uint4 u[sizeof(T) / 2];
    template <bool WHOLE> __device__ __forceinline__ void load(const T *p, int64_t left, bool wide)
    {
        if (WHOLE || (wide && left >= 8)) {
#pragma unroll
            for (int i = 0; i < int(sizeof(T) / 2); ++i) u[i] = load_now(reinterpret_cast<const uint4 *>(p) + i);
        } else {
            T *e = reinterpret_cast<T *>(u);
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = i < left ? p[i] : from_f32<T>(0.0f);
        }
    }
    // Lets the compiler convert them again instead of keeping all of them as floats.
    __device__ __forceinline__ void again()
    {
#pragma unroll
        for (int i = 0; i < int(sizeof(T) / 2); ++i) asm volatile("" : "+r"(u[i].x), "+r"(u[i].y), "+r"(u[i].z), "+r"(u[i].w));
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        const T *e = reinterpret_cast<const T *>(u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
    }
};

// Two 16-bit elements.
template <class T> struct Two {};
template <> struct Two<__half> {
    using type = __half2;
    static __device__ __forceinline__ type zero() { return __floats2half2_rn(0.0f, 0.0f); }
};
template <> struct Two<__nv_bfloat16> {
    using type = __nv_bfloat162;
    static __device__ __forceinline__ type zero() { return __floats2bfloat162_rn(0.0f, 0.0f); }
};

// The largest magnitude (fmaxf, as __hmax2, passes over NaN).
__device__ __forceinline__ float largest(const float (&v)[8])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
}
// Eight values times 2^(127 - exponent) as 8-bit codes.  An infinity is stored as NaN like NaN itself: neither
// turns finite, e4m3 has no infinity.  infinite: whether there may be one.
template <bool E5M2, class Exponent> __device__ __forceinline__ uint2 codes(const float (&v)[8], bool infinite, Exponent exponent)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 by = make_float2(power(254u - exponent(2 * i)), power(254u - exponent(2 * i + 1)));
        const float2 f = __fmul2_rn(make_float2(v[2 * i], v[2 * i + 1]), by);
        w[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, E5M2 ? __NV_E5M2 : __NV_E4M3);
    }
    if (__builtin_expect(infinite, 0)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (fabsf(v[2 * i]) > FLT_MAX) w[i] |= 0x7fu;
            if (fabsf(v[2 * i + 1]) > FLT_MAX) w[i] |= 0x7f00u;
        }
    }
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

template <bool WHOLE> __device__ __forceinline__ void put_codes(uint8_t *q, uint2 w, int64_t left)
{
    if (WHOLE || left >= 8) {
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
    int col_blocks, wide;
};

struct QuantizeSpace {
    float column_max[16][128];
    uint32_t column_exponent[128];
    float warp_max[kThreads / 32];
};

// One tile.  WHOLE: it lies inside the matrix and its rows are read in 16-byte pieces.
template <class T, int MODE, int I, bool E5M2, bool WHOLE>
__device__ __forceinline__ void quantize_tile(const QuantizeParams &p, int64_t rb, int64_t cb, QuantizeSpace &space)
{
    constexpr int kTop = E5M2 ? 15 : 8;
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
    const int64_t r0 = rb * (16 * I) + y, c = cb * 128 + x * 8, left = p.cols - c;
    const T *src = static_cast<const T *>(p.X) + r0 * p.ldx + c;
    Piece<T> piece[I];
#pragma unroll
    for (int i = 0; i < I; ++i)
        piece[i].template load<WHOLE>(src + int64_t(16 * i) * p.ldx, WHOLE || r0 + 16 * i < p.rows ? left : 0, p.wide);
    auto inside = [&](int i) { return WHOLE || (r0 + 16 * i < p.rows && left > 0); };
    // an infinity in this thread's pieces shows in the first look, and is left out in a second one
    float row[I], column[8];
    bool infinite = false;
    if constexpr (sizeof(T) == 2) {  // maxima of two elements at once, in their own type
        using T2 = typename Two<T>::type;
        const T2 zero = Two<T>::zero();
        T2 most[4] = {zero, zero, zero, zero};
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const T2 *e = reinterpret_cast<const T2 *>(piece[i].u);
            T2 m = zero;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const T2 a = __habs2(e[j]);
                m = __hmax2(m, a);
                if ((MODE & kColumns) != 0) most[j] = __hmax2(most[j], a);
            }
            row[i] = fmaxf(to_f32(m.x), to_f32(m.y));
            infinite = infinite || row[i] > FLT_MAX;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) column[j] = to_f32(j & 1 ? most[j / 2].y : most[j / 2].x);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) column[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            float v[8];
            piece[i].get(v);
            row[i] = largest(v);
            infinite = infinite || row[i] > FLT_MAX;
            if ((MODE & kColumns) != 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) column[j] = fmaxf(column[j], fabsf(v[j]));
            }
        }
    }
    if (__builtin_expect(infinite, 0)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) column[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            float v[8];
            piece[i].get(v);
            row[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float a = fabsf(v[j]) <= FLT_MAX ? fabsf(v[j]) : 0.0f;
                row[i] = fmaxf(row[i], a);
                column[j] = fmaxf(column[j], a);
            }
        }
    }
    if constexpr ((MODE & kColumns) != 0) {
        float4 *to = reinterpret_cast<float4 *>(&space.column_max[y][x * 8]);
        to[0] = make_float4(column[0], column[1], column[2], column[3]);
        to[1] = make_float4(column[4], column[5], column[6], column[7]);
    }
    if constexpr ((MODE & kRows) != 0) {
        // Lanes that are o apart share what is left of their rows: each hands the other one half and keeps the
        // maxima of the other half, so that with eight rows lane x ends with row 4 (x / 8 % 2) + 2 (x / 4 % 2) +
        // x / 2 % 2 and one exponent to find, which the others then ask it for (16 exchanges a thread, not 32).
        float most[I];
#pragma unroll
        for (int i = 0; i < I; ++i) most[i] = row[i];
#pragma unroll
        for (int o = 8, n = I / 2; o > 0; o >>= 1, n /= 2) {
            if (n > 0) {
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const float mine = x & o ? most[i + n] : most[i], theirs = x & o ? most[i] : most[i + n];
                    most[i] = fmaxf(mine, __shfl_xor_sync(kFull, theirs, o));
                }
            } else {
                most[0] = fmaxf(most[0], __shfl_xor_sync(kFull, most[0], o));
            }
        }
        static_assert(I == 8 || I == 1, "the lane of a row");
        const uint32_t exponent = scale_exponent(most[0], kTop);
        const int64_t mine = I == 1 ? r0 : r0 + 16 * ((x >> 3) * 4 + (x >> 2 & 1) * 2 + (x >> 1 & 1));
        if ((I == 1 ? x : x & 1) == 0 && (WHOLE || mine < p.rows)) p.s.at[mine * p.s.row + cb * p.s.col] = power(exponent);
        uint8_t *q = p.Q + r0 * p.ldq + c;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const uint32_t e = I == 1 ? exponent : __shfl_sync(kFull, exponent, (i >> 2) * 8 + (i >> 1 & 1) * 4 + (i & 1) * 2, 16);
            float v[8];
            if (sizeof(T) == 2) piece[i].again();
            piece[i].get(v);
            const uint2 w = codes<E5M2>(v, infinite, [=](int) { return e; });
            if (inside(i)) put_codes<WHOLE>(q + int64_t(16 * i) * p.ldq, w, left);
        }
    }
    if constexpr ((MODE & kTiles) != 0) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < I; ++i) m = fmaxf(m, row[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        if ((threadIdx.x & 31) == 0) space.warp_max[threadIdx.x >> 5] = m;
        __syncthreads();
        m = space.warp_max[0];
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) m = fmaxf(m, space.warp_max[i]);
        const uint32_t e = scale_exponent(m, kTop);
        if (threadIdx.x == 0) p.s.at[rb * p.s.row + cb * p.s.col] = power(e);
        uint8_t *q = p.Q + r0 * p.ldq + c;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            float v[8];
            if (sizeof(T) == 2) piece[i].again();
            piece[i].get(v);
            const uint2 w = codes<E5M2>(v, infinite, [=](int) { return e; });
            if (inside(i)) put_codes<WHOLE>(q + int64_t(16 * i) * p.ldq, w, left);
        }
    }
    if constexpr ((MODE & kColumns) != 0) {
        __syncthreads();
        if (threadIdx.x < 128) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) m = fmaxf(m, space.column_max[i][threadIdx.x]);
            const uint32_t e = scale_exponent(m, kTop);
            space.column_exponent[threadIdx.x] = e;
            const int64_t col = cb * 128 + threadIdx.x;
            if (WHOLE || col < p.cols) p.sc.at[rb * p.sc.row + col * p.sc.col] = power(e);
        }
        __syncthreads();
        uint32_t e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = space.column_exponent[x * 8 + j];
        uint8_t *q = p.Qc + r0 * p.ldqc + c;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            float v[8];
            if (sizeof(T) == 2) piece[i].again();
            piece[i].get(v);
            const uint2 w = codes<E5M2>(v, infinite, [&](int j) { return e[j]; });
            if (inside(i)) put_codes<WHOLE>(q + int64_t(16 * i) * p.ldqc, w, left);
        }
    }
}

// Thread (x, y) = (t % 16, t / 16): 8 columns of the rows y, y + 16, .. of a tile of 16 * I rows.  MODE: the
// sum of the ways.  Blocks of 1 x 128 alone do not need a tile's height: few rows take I = 1, for more CTAs.
template <class T, int MODE, int I, bool E5M2>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 2 : 3) quantize_kernel(const __grid_constant__ QuantizeParams p)
{
    __shared__ QuantizeSpace space;
    chain_wait();
    const int64_t rb = blockIdx.x / unsigned(p.col_blocks), cb = blockIdx.x % unsigned(p.col_blocks);
    if (p.wide && (rb + 1) * 16 * I <= p.rows && (cb + 1) * 128 <= p.cols) quantize_tile<T, MODE, I, E5M2, true>(p, rb, cb, space);
    else quantize_tile<T, MODE, I, E5M2, false>(p, rb, cb, space);
}

template <class T, bool E5M2> cudaError_t quantize(const QuantizeArgs &a, cudaStream_t stream)
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
    p.wide = reinterpret_cast<uintptr_t>(a.X) % 16 == 0 && a.ldx * int64_t(sizeof(T)) % 16 == 0;
    const int64_t blocks = (a.cols + 127) / 128;
    p.col_blocks = int(blocks);
    const bool rows_alone = a.Qc == nullptr && a.s.row_shift == 0;
    // few rows: 16 a CTA (64 x 4096 on 128 CTAs instead of 32)
    const bool few = rows_alone && ((a.rows + 127) / 128) * blocks < 304;
    const int64_t height = few ? 16 : 128, grid = (a.rows + height - 1) / height * blocks;
    if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    const dim3 g{unsigned(grid)};
    if (few) return launch_chained(quantize_kernel<T, kRows, 1, E5M2>, g, kThreads, 0, 1, stream, p);
    if (rows_alone) return launch_chained(quantize_kernel<T, kRows, 8, E5M2>, g, kThreads, 0, 1, stream, p);
    if (a.Q == nullptr) return launch_chained(quantize_kernel<T, kColumns, 8, E5M2>, g, kThreads, 0, 1, stream, p);
    if (a.Qc == nullptr) return launch_chained(quantize_kernel<T, kTiles, 8, E5M2>, g, kThreads, 0, 1, stream, p);
    return launch_chained(quantize_kernel<T, kRows + kColumns, 8, E5M2>, g, kThreads, 0, 1, stream, p);
}
template <class T> cudaError_t quantize(const QuantizeArgs &a, cudaStream_t stream)
{
    return a.q_type == GEMM_TYPE_E5M2 ? quantize<T, true>(a, stream) : quantize<T, false>(a, stream);
}

// Eight values to a boundary of as many.  fp32: one 32-byte store, since two of 16 each leave half sectors to L2
// (16384 x 4096: 67 us).
template <class Y> __device__ __forceinline__ void store_piece(Y *to, const float (&f)[8])
{
    if constexpr (sizeof(Y) == 4)
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]),
                     "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                     : "memory");
    else
        store8<Y>(to, f);
}

// Thread (x, y) of a CTA: 8 columns of the rows y, y + 16, .. of a tile of 128 x 128, whose scales are one a
// row, one a column or one; eight pieces in flight.
template <class Y, bool E5M2>
__global__ void __launch_bounds__(kThreads, 4)
dequantize_kernel(int64_t rows, int64_t cols, unsigned col_blocks, const uint8_t *Q, int64_t ldq, const __grid_constant__ Scales s, Y *y,
                  int64_t ldy, int wide)
{
    chain_wait();
    const int64_t rb = blockIdx.x / col_blocks, cb = blockIdx.x % col_blocks;
    const int64_t r0 = rb * 128 + (threadIdx.x >> 4), c = cb * 128 + (threadIdx.x & 15) * 8, left = cols - c;
    if (left <= 0) return;
    uint2 w[8];
    float row[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 16 * i;
        w[i] = make_uint2(0u, 0u);
        row[i] = 1.0f;
        if (r >= rows) continue;
        const uint8_t *q = Q + r * ldq + c;
        if (left >= 8) {
            w[i] = load_now(reinterpret_cast<const uint2 *>(q));
        } else {
            for (int j = 0; j < left; ++j) (j < 4 ? w[i].x : w[i].y) |= uint32_t(q[j]) << (8 * (j & 3));
        }
        if (s.col_shift != 0) row[i] = load_now(s.at + (r >> s.row_shift) * s.row + cb * s.col);
    }
    float column[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) column[j] = s.col_shift == 0 && j < left ? load_now(s.at + rb * s.row + (c + j) * s.col) : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 16 * i;
        if (r >= rows) break;
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint16_t two = uint16_t((j < 2 ? w[i].x : w[i].y) >> (16 * (j & 1)));
            const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, E5M2 ? __NV_E5M2 : __NV_E4M3)));
            f[2 * j] = v.x * row[i] * column[2 * j];  // one of the two scales is 1
            f[2 * j + 1] = v.y * row[i] * column[2 * j + 1];
        }
        Y *to = y + r * ldy + c;
        if (wide && left >= 8) {
            store_piece<Y>(to, f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < left) to[j] = from_f32<Y>(f[j]);
        }
    }
}

template <class Y>
cudaError_t dequantize(int q_type, int64_t rows, int64_t cols, const void *Q, int64_t ldq, const Scales &s, void *y, int64_t ldy,
                       cudaStream_t stream)
{
    const int wide = reinterpret_cast<uintptr_t>(y) % (8 * sizeof(Y)) == 0 && ldy % 8 == 0;
    const int64_t blocks = (cols + 127) / 128, grid = (rows + 127) / 128 * blocks;
    if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    return launch_chained(q_type == GEMM_TYPE_E5M2 ? dequantize_kernel<Y, true> : dequantize_kernel<Y, false>, dim3(unsigned(grid)), kThreads,
                          0, 1, stream, rows, cols, unsigned(blocks), static_cast<const uint8_t *>(Q), ldq, s, static_cast<Y *>(y), ldy, wide);
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
