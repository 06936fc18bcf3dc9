// The orthogonalised update: its C entry point, the plan of its steps, and the row kernels around its
// products (semantics: include/gemm_gb300.h; the products: orthogonal_tcgen05.cu).
//
// Every iterate is held as powers of two times fp16 values, whose exponents the host chooses for each step
// from a bound on the singular values: on [0, r] the polynomial's largest magnitude bounds the next r.
//
// The row kernels are bound by memory: 4096 x 4096 fp32 (GB300): sum of squares 15.6 us (4.3 TB/s), parts 24 (5.6).
// The partial sums are a fixed number whatever the stack, and added in order: a result is the same from run to
// run and in any stack.
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>

#include "orthogonal_internal.h"

namespace gemm {
namespace {

constexpr int kThreads = 256;
constexpr unsigned kFull = 0xffffffffu;
constexpr int64_t kMaxSide = (int64_t(1) << 20) - 1;
constexpr int64_t kMaxLd = int64_t(1) << 35;
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int kMaxSteps = 64;

// ------------------------------------------------------------------ norm
// Squares of values far from 1 leave fp32's range: values below 2^-40 and above 2^40 are summed apart,
// moved by 2^86.  (All three stay in range for 2^33 elements.  Doubles from the partial sums on cost 1.2 us in
// either kernel.)
struct Squares {
    float low = 0.0f, mid = 0.0f, high = 0.0f;
    // Eight values, together in the common case.
    __device__ __forceinline__ void add(const float (&v)[8])
    {
        float least = FLT_MAX, most = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = fabsf(v[i]);
            least = fminf(least, a == 0.0f ? 1.0f : a);
            most = fmaxf(most, a);
        }
        if (least >= 0x1p-40f && most <= 0x1p40f) {  // NaN too
            float a = v[0] * v[0], b = v[1] * v[1];
#pragma unroll
            for (int i = 2; i < 8; i += 2) {
                a = fmaf(v[i], v[i], a);
                b = fmaf(v[i + 1], v[i + 1], b);
            }
            mid += a + b;
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = fabsf(v[i]);
            if (a < 0x1p-40f) low = fmaf(a * 0x1p86f, a * 0x1p86f, low);
            else if (a > 0x1p40f) high = fmaf(a * 0x1p-86f, a * 0x1p-86f, high);
            else mid = fmaf(v[i], v[i], mid);
        }
    }
    __device__ __forceinline__ void add_lanes()
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            low += __shfl_xor_sync(kFull, low, o);
            mid += __shfl_xor_sync(kFull, mid, o);
            high += __shfl_xor_sync(kFull, high, o);
        }
    }
    __device__ __forceinline__ void add(const float4 &v) { low += v.x, mid += v.y, high += v.z; }
};

// Thread: every so many 16-byte pieces of eight elements, four in flight.  I: what the pieces are counted in.
template <class T, class I>
__global__ void __launch_bounds__(kThreads)
squares_kernel(int64_t rows, int64_t cols, const T *G, int64_t ld, int64_t stride, int wide, float4 *partial)
{
    __shared__ float4 sums[kThreads / 32];
    chain_wait();
    const T *g = G + int64_t(blockIdx.y) * stride;
    Squares s;
    const I pieces = I((cols + 7) / 8), total = I(rows) * pieces, step = I(gridDim.x) * kThreads;
    for (I i0 = I(blockIdx.x) * kThreads + threadIdx.x; i0 < total; i0 += 4 * step) {
        float v[4][8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const I i = i0 + I(q) * step, r = i / pieces;
            const int64_t c = int64_t(i - r * pieces) * 8;
            if (i < total && wide && c + 8 <= cols) {
                load8<T>(g + int64_t(r) * ld + c, v[q]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[q][j] = i < total && c + j < cols ? to_f32(g[int64_t(r) * ld + c + j]) : 0.0f;
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) s.add(v[q]);
    }
    s.add_lanes();
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = make_float4(s.low, s.mid, s.high, 0.0f);
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) s.add(sums[i]);
        partial[int64_t(blockIdx.y) * kNormBlocks + blockIdx.x] = make_float4(s.low, s.mid, s.high, 0.0f);
    }
}

struct Norm {
    int exponent;  // 2^exponent <= norm < 2^(exponent + 1)
    float unit;    // 2^exponent / norm, NaN where the norm is no finite number
};
__device__ __forceinline__ Norm norm_of(const Squares &s, float eps)
{
    // the norm is sqrt(square) * 2^moved; what the sums of smaller values lose on the way is far below its rounding
    float square = s.low;
    int moved = -86;
    if (!(s.high == 0.0f)) {  // an infinity and NaN too
        square = fmaf(s.mid * 0x1p-86f, 0x1p-86f, s.high);
        moved = 86;
    } else if (s.mid > 0.0f || (eps >= 0x1p14f)) {
        square = fmaf(s.low * 0x1p-86f, 0x1p-86f, s.mid);
        moved = 0;
    }
    if (!(s.mid >= 0.0f && s.low >= 0.0f)) square = s.mid + s.low;  // NaN
    // a quarter of both, so that their sum stays finite
    const float by = moved == 86 ? 0x1p-88f : moved == 0 ? 0x1p-2f : 0x1p84f, norm = fmaf(sqrtf(square), 0.25f, eps * by);
    if (!(norm <= FLT_MAX)) return Norm{0, __uint_as_float(0x7fffffffu)};
    if (norm == 0.0f) return Norm{0, 1.0f};
    int e;
    const float m = frexpf(norm, &e);  // in [1/2, 1)
    return Norm{e + 1 + moved, 0.5f / m};
}

__device__ __forceinline__ float two_to(int e) { return __uint_as_float(uint32_t(max(-126, min(127, e)) + 127) << 23); }

// x = high + low to 22 bits, down to fp16's smallest step, 2^-24.
__device__ __forceinline__ void parts(float x, __half &high, __half &low)
{
    high = __float2half_rn(x);
    low = __float2half_rn(x - __half2float(high));
}

// Tiles of 64 x 64 elements of G to the parts of X, TURN: transposed through shared memory.
template <class T, bool TURN>
__global__ void __launch_bounds__(kThreads)
split_kernel(int64_t rows, int64_t cols, const T *G, int64_t ld, int64_t stride, int wide, int blocks, const float4 *partial, float eps,
             __half *X, int64_t ldx, int64_t n, int64_t part_stride, float *unit)
{
    __shared__ float tile[TURN ? 64 : 1][65];
    __shared__ float factor[2];
    chain_wait();
    const int64_t which = blockIdx.z;
    const T *g = G + which * stride;
    __half *x = X + which * n * ldx;
    const int64_t r0 = int64_t(blockIdx.y) * 64, c0 = int64_t(blockIdx.x) * 64;
    const int piece = threadIdx.x & 7, line = threadIdx.x >> 3;  // 8 elements of one of 32 rows
    float v[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t r = r0 + line + 32 * h, c = c0 + piece * 8;
        if (r < rows && wide && c + 8 <= cols) {
            load8<T>(g + r * ld + c, v[h]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[h][j] = r < rows && c + j < cols ? to_f32(g[r * ld + c + j]) : 0.0f;
        }
    }
    if (threadIdx.x < 32) {
        Squares s;
        for (int i = threadIdx.x; i < blocks; i += 32) s.add(partial[which * kNormBlocks + i]);
        s.add_lanes();
        if (threadIdx.x == 0) {
            const Norm norm = norm_of(s, eps);
            const int e = kFirstScale - norm.exponent;  // in two factors, which fp32 holds
            factor[0] = two_to(e / 2);
            factor[1] = two_to(e - e / 2);
            if (blockIdx.x == 0 && blockIdx.y == 0) unit[which] = norm.unit;
        }
    }
    __syncthreads();
    const float f0 = factor[0], f1 = factor[1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t r = r0 + line + 32 * h, c = c0 + piece * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[h][j] = v[h][j] * f0 * f1;
        if (TURN) {
#pragma unroll
            for (int j = 0; j < 8; ++j) tile[line + 32 * h][piece * 8 + j] = v[h][j];
        } else if (r < rows && c < cols) {  // up to the padded row's end
            __half high[8], low[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) parts(v[h][j], high[j], low[j]);
            *reinterpret_cast<uint4 *>(x + r * ldx + c) = *reinterpret_cast<const uint4 *>(high);
            *reinterpret_cast<uint4 *>(x + part_stride + r * ldx + c) = *reinterpret_cast<const uint4 *>(low);
        }
    }
    if constexpr (TURN) {
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 64; h += 32) {
            const int64_t r = c0 + line + h, c = r0 + piece * 8;  // of X
            if (r >= cols || c >= rows) continue;
            __half high[8], low[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) parts(tile[piece * 8 + j][line + h], high[j], low[j]);
            *reinterpret_cast<uint4 *>(x + r * ldx + c) = *reinterpret_cast<const uint4 *>(high);
            *reinterpret_cast<uint4 *>(x + part_stride + r * ldx + c) = *reinterpret_cast<const uint4 *>(low);
        }
    }
}

template <class T> cudaError_t normalise(const OrthogonalArgs &a, const OrthogonalLayout &l, cudaStream_t stream)
{
    char *w = static_cast<char *>(a.work);
    float4 *partial = reinterpret_cast<float4 *>(w + l.partial);
    const T *G = static_cast<const T *>(a.G);
    const int wide = reinterpret_cast<uintptr_t>(G) % 16 == 0 && a.ldg * int64_t(sizeof(T)) % 16 == 0 &&
                     (a.count == 1 || a.strideg * int64_t(sizeof(T)) % 16 == 0);
    const int64_t pieces = a.rows * ((a.cols + 7) / 8), wanted = (pieces + 4 * kThreads - 1) / (4 * kThreads);
    const int blocks = int(wanted < kNormBlocks ? wanted : kNormBlocks);  // whatever the count: a stack gives each matrix's own result
    const dim3 parts(unsigned(blocks), unsigned(a.count));
    // 32-bit places leave room for the last step beyond the end
    cudaError_t e = pieces < (int64_t(1) << 31) ? launch_chained(squares_kernel<T, unsigned>, parts, kThreads, 0, 1, stream, a.rows, a.cols, G,
                                                                 a.ldg, a.strideg, wide, partial)
                                                : launch_chained(squares_kernel<T, int64_t>, parts, kThreads, 0, 1, stream, a.rows, a.cols, G,
                                                                 a.ldg, a.strideg, wide, partial);
    if (e != cudaSuccess) return e;
    const dim3 grid{unsigned((a.cols + 63) / 64), unsigned((a.rows + 63) / 64), unsigned(a.count)};
    return launch_chained(a.rows > a.cols ? split_kernel<T, true> : split_kernel<T, false>, grid, kThreads, 0, 1, stream, a.rows, a.cols,
                          G, a.ldg, a.strideg, wide, blocks, static_cast<const float4 *>(partial), a.eps,
                          reinterpret_cast<__half *>(w + l.x[0]), l.ldk, l.n, l.count * l.n * l.ldk,
                          reinterpret_cast<float *>(w + l.unit));
}

// ------------------------------------------------------------------ bounds of a step
// The largest |a s + b s^3 + c s^5| on [0, r].
double largest_value(double a, double b, double c, double r)
{
    auto p = [&](double s) { return std::fabs(s * (a + s * s * (b + s * s * c))); };
    double most = p(r);
    auto at = [&](double t) {  // t = s^2, a root of a + 3 b t + 5 c t^2
        if (t > 0.0 && t < r * r) most = std::fmax(most, p(std::sqrt(t)));
    };
    if (c != 0.0) {
        const double q = 9.0 * b * b - 20.0 * a * c;
        if (q >= 0.0) {
            at((-3.0 * b + std::sqrt(q)) / (10.0 * c));
            at((-3.0 * b - std::sqrt(q)) / (10.0 * c));
        }
    } else if (b != 0.0) {
        at(-a / (3.0 * b));
    }
    return most;
}
// The largest |b t + c t^2| on [0, r^2]: of b A + c A^2.
double largest_inner(double b, double c, double r)
{
    const double end = r * r;
    double most = std::fabs(b * end + c * end * end);
    if (c != 0.0 && -b / (2.0 * c) > 0.0 && -b / (2.0 * c) < end) most = std::fmax(most, b * b / (4.0 * std::fabs(c)));
    return most;
}
// The power of two that brings values up to `bound` close to, and not over, 60000 in fp16.  The iterates' bounds are
// kLeastBound or more, so those of A are its square or more; for b A + c A^2, which may vanish, kLeastResult stands for
// less: what its parts then lose is below 2^-100, far below any result.  Two such scales' product and its inverse are
// in fp32's range.
constexpr double kLeastBound = 0x1p-20, kLeastResult = 0x1p-60;
float scale_for(double bound)
{
    int e;
    std::frexp(60000.0 / std::fmax(bound, kLeastResult), &e);
    return float(std::ldexp(1.0, e - 1));
}

bool is_type(int t) { return t == GEMM_TYPE_F32 || t == GEMM_TYPE_F16 || t == GEMM_TYPE_BF16; }
bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

gemm_status_t check_sides(int64_t count, int64_t rows, int64_t cols)
{
    if (count < 0 || rows < 0 || cols < 0) return GEMM_ERR_INVALID_VALUE;
    if (count > 65535 || rows > kMaxSide || cols > kMaxSide) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

}  // namespace

OrthogonalLayout orthogonal_layout(int64_t count, int64_t rows, int64_t cols)
{
    OrthogonalLayout l{};
    l.n = rows < cols ? rows : cols;
    l.k = rows < cols ? cols : rows;
    l.count = count;
    l.ldk = (l.k + 63) / 64 * 64;
    l.ldn = (l.n + 63) / 64 * 64;
    auto take = [&](int64_t bytes) {
        const int64_t at = l.bytes;
        l.bytes += (bytes + 255) / 256 * 256;
        return at;
    };
    for (int i = 0; i < 2; ++i) l.x[i] = take(2 * count * l.n * l.ldk * 2);
    l.e = take(2 * count * l.n * l.ldn * 2);
    l.f = take(2 * count * l.n * l.ldn * 2);
    l.dd = take(count * l.ldn * 4);
    l.df = take(count * l.ldn * 4);
    l.unit = take(count * 4);
    l.partial = take(count * kNormBlocks * int64_t(sizeof(float4)));
    return l;
}

cudaError_t launch_normalise(const OrthogonalArgs &a, const OrthogonalLayout &l, cudaStream_t stream)
{
    if (a.type == GEMM_TYPE_F32) return normalise<float>(a, l, stream);
    if (a.type == GEMM_TYPE_F16) return normalise<__half>(a, l, stream);
    return normalise<__nv_bfloat16>(a, l, stream);
}

}  // namespace gemm

using namespace gemm;

extern "C" {

int64_t gemm_orthogonalize_work_bytes(int64_t count, int64_t rows, int64_t cols)
{
    if (check_sides(count, rows, cols) != GEMM_OK || count == 0 || rows == 0 || cols == 0) return 0;
    return orthogonal_layout(count, rows, cols).bytes;
}

gemm_status_t gemm_orthogonalize(gemm_type_t type, gemm_type_t y_type, int64_t count, int64_t rows, int64_t cols, const void *G, int64_t ldg,
                                 int64_t strideG, int steps, const float *coefficients, float eps, void *Y, int64_t ldy,
                                 int64_t strideY, void *work, void *stream)
{
    if (!is_type(type) || !is_type(y_type) || steps < 1 || coefficients == nullptr ||
        !(eps >= 0.0f && eps <= FLT_MAX) || strideG < 0 || strideY < 0)
        return GEMM_ERR_INVALID_VALUE;
    gemm_status_t s = check_sides(count, rows, cols);
    if (s != GEMM_OK) return s;
    if (ldg < (cols > 1 ? cols : 1) || ldy < (cols > 1 ? cols : 1)) return GEMM_ERR_INVALID_VALUE;
    if (ldg > kMaxLd || ldy > kMaxLd || strideG > kMaxStride || strideY > kMaxStride || steps > kMaxSteps) return GEMM_ERR_UNSUPPORTED;
    // the singular values stay within r, with some room for rounding
    OrthogonalStep plan[kMaxSteps];
    double r = 1.0;
    for (int i = 0; i < steps; ++i) {
        const float a = coefficients[3 * i], b = coefficients[3 * i + 1], c = coefficients[3 * i + 2];
        if (!(std::fabs(a) <= 1e4f && std::fabs(b) <= 1e4f && std::fabs(c) <= 1e4f)) return GEMM_ERR_UNSUPPORTED;
        OrthogonalStep &p = plan[i];
        p = OrthogonalStep{a, b, c, i == 0 ? float(1 << kFirstScale) : plan[i - 1].next_scale, scale_for(r * r),
                           scale_for(1.02 * largest_inner(b, c, r)), 1.0f};
        r = 1.02 * largest_value(a, b, c, r);
        if (!(r <= 1e4) || (i + 1 < steps ? r < kLeastBound : r > 0.0 && r < kLeastResult)) return GEMM_ERR_UNSUPPORTED;
        p.next_scale = scale_for(r);
    }
    if (count == 0 || rows == 0 || cols == 0) return GEMM_OK;
    if (G == nullptr || Y == nullptr || work == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (count > 1 && strideY < (rows - 1) * ldy + cols) return GEMM_ERR_INVALID_VALUE;
    if (!aligned(G, type == GEMM_TYPE_F32 ? 4 : 2) || !aligned(Y, 16) || ldy % 8 != 0 || (count > 1 && strideY % 8 != 0) ||
        !aligned(work, 256))
        return GEMM_ERR_MISALIGNED;
    DeviceInfo dev;
    if (!current_device(dev) || dev.cc_major != 10 || dev.cc_minor != 3) return GEMM_ERR_NO_DEVICE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const OrthogonalArgs a{type, y_type, count, rows, cols, G, ldg, strideG, Y, ldy, strideY, eps, work};
    const OrthogonalLayout l = orthogonal_layout(count, rows, cols);
    cudaError_t e = launch_normalise(a, l, st);
    if (e == cudaSuccess) e = launch_orthogonal_steps(dev, a, l, plan, steps, st);
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // extern "C"
