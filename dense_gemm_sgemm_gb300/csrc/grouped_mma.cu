// Products with few rows per weight matrix: a decoding step's experts, a decoding step's linear
// layer with adapters, and the inner product of the adapters (semantics: include/gemm_gb300.h).
//
// With a handful of rows a product is bound by reading its weights once: at 8 rows a weight matrix
// brings 8 flops per byte, where the tensor cores could do 280.  So the weights never touch shared
// memory.  A warp computes D[feature][token] = W X^T with mma.sync m16n8k16: the weight rows are
// the m side (16 or 32 rows a warp), up to 8 * NT tokens the n side.  The order of k inside a
// product is free as long as both operands agree, so lane (g, t) loads 16 contiguous bytes --
// W[g][8 t .. 8 t + 7] of a 32-wide k step, X likewise -- and the four registers of the load are
// the fragments of two MMAs: every weight byte goes from global memory to its register in one
// 16-byte load, several steps ahead of use.  K is split over warps of the CTA where rows alone do
// not fill the machine; their partial sums meet in shared memory in a fixed order.
#include <cuda_runtime.h>

#include <type_traits>

#include "routed_internal.h"

namespace gemm {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
// Floats between tokens of a warp's partial tile of MT x 16 rows: 8 t + g, no bank twice.
template <int MT> constexpr int kRowStride = MT <= 2 ? 36 : 68;
constexpr unsigned kFull = 0xffffffffu;

// Rows that one warp reads once: no line of L1 for them.
__device__ __forceinline__ uint4 load_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// acc[mt][nt] += W X^T over k in [kb, ke) (kb a multiple of 32, ke one or K).  w[mt][h]: the row of
// this lane's group in the lower and upper half of tile mt; x[nt]: the token row of this lane's
// group, NULL for a column of zeros.
//
// FLIGHT: registers of loads in flight, 64 where a CTA's 16 warps leave a thread 128 registers.
template <class T, int MT, int NT, int FLIGHT = 96>
__device__ __forceinline__ void warp_product(const T *const (&w)[MT][2], const T *const (&x)[NT], int64_t kb,
                                             int64_t ke, int64_t K, int lane, float (&acc)[MT][NT][4])
{
    constexpr int U = MT * 2 * 4 * 4 + NT * 4 * 4 <= FLIGHT ? 4 : MT * 2 * 4 * 2 + NT * 4 * 2 <= FLIGHT ? 2 : 1;
    const int t8 = (lane & 3) * 8;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    auto multiply = [&](const uint4 (&a)[MT][2], const uint4 (&b)[NT]) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma_16816<T>(acc[m][n], a[m][0].x, a[m][1].x, a[m][0].y, a[m][1].y, b[n].x, b[n].y);
                mma_16816<T>(acc[m][n], a[m][0].z, a[m][1].z, a[m][0].w, a[m][1].w, b[n].z, b[n].w);
            }
    };
    int64_t k = kb;
    for (; k + 32 * U <= ke; k += 32 * U) {
        uint4 a[U][MT][2], b[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) a[u][m][h] = load_stream(w[m][h] + k + 32 * u + t8);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                b[u][n] = x[n] != nullptr ? __ldg(reinterpret_cast<const uint4 *>(x[n] + k + 32 * u + t8)) : zero;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) multiply(a[u], b[u]);
    }
    for (; k < ke; k += 32) {
        uint4 a[MT][2], b[NT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) a[m][h] = load_tail(w[m][h], k + t8, K);
#pragma unroll
        for (int n = 0; n < NT; ++n) b[n] = x[n] != nullptr ? load_tail(x[n], k + t8, K) : zero;
        multiply(a, b);
    }
}

// Partial tile of a warp to shared memory as [token][feature row].
template <int MT, int NT>
__device__ __forceinline__ void put_partial(float *part, const float (&acc)[MT][NT][4], int lane)
{
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                part[(n * 8 + 2 * t + (c & 1)) * kRowStride<MT> + m * 16 + g + 8 * (c >> 1)] = acc[m][n][c];
}

__device__ __forceinline__ int32_t clamp_to(int32_t v, int64_t hi) { return v < 0 ? 0 : v > hi ? int32_t(hi) : v; }

// First position and rows of the i-th group that has rows; false when there are fewer.
__device__ __forceinline__ bool nonempty_group(const GroupedArgs &a, int i, int lane, int &group, int &first, int &rows)
{
    if (a.offsets == nullptr) {
        group = 0;
        first = 0;
        rows = int(a.y_rows);
        return i == 0 && rows > 0;
    }
    int seen = 0;
    for (int e0 = 0; e0 < a.groups; e0 += 32) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < a.groups) {
            lo = clamp_to(__ldg(a.offsets + e), a.y_rows);
            hi = clamp_to(__ldg(a.offsets + e + 1), a.y_rows);
        }
        const unsigned has = __ballot_sync(kFull, hi > lo);
        const int n = __popc(has);
        if (seen + n > i) {
            const int at = __fns(has, 0, i - seen + 1);
            group = e0 + at;
            first = __shfl_sync(kFull, lo, at);
            rows = __shfl_sync(kFull, hi, at) - first;
            return true;
        }
        seen += n;
    }
    return false;
}

// low[q] += B_a[feature] . inner[position] of output q, which `place` locates (false: no such output).
// The adapter of the position, then its row of B: two latencies, so COUNT outputs share them.
// Outputs without an adapter read the first one's and take nothing from it.
template <class T, int COUNT, class Place>
__device__ __forceinline__ void add_adapters(const GroupedArgs &a, float (&low)[COUNT], Place place)
{
    const T *b[COUNT];
    const float *inner[COUNT];
    bool has[COUNT];
#pragma unroll
    for (int q = 0; q < COUNT; ++q) {
        int64_t p, feat;
        has[q] = place(q, p, feat);
        if (!has[q]) p = feat = 0;
        int which = __ldcg(a.ad.which + p);
        has[q] = has[q] && unsigned(which) < unsigned(a.ad.count);
        if (!has[q]) which = 0;
        b[q] = static_cast<const T *>(a.ad.b) + int64_t(which) * a.ad.strideb + feat * a.ad.ldb;
        inner[q] = static_cast<const float *>(a.ad.inner) + p * a.ad.rank;
    }
    const bool whole = a.ad.rank % 8 == 0;
    for (int j = 0; j < a.ad.rank; j += 8) {
        uint4 e[COUNT];
        float x[COUNT][8];
#pragma unroll
        for (int q = 0; q < COUNT; ++q) {
            if (whole) {
                e[q] = __ldg(reinterpret_cast<const uint4 *>(b[q] + j));
                reinterpret_cast<float4 *>(x[q])[0] = __ldcg(reinterpret_cast<const float4 *>(inner[q] + j));
                reinterpret_cast<float4 *>(x[q])[1] = __ldcg(reinterpret_cast<const float4 *>(inner[q] + j) + 1);
            } else {
                e[q] = load_tail(b[q], j, a.ad.rank);
#pragma unroll
                for (int c = 0; c < 8; ++c) x[q][c] = j + c < a.ad.rank ? __ldcg(inner[q] + j + c) : 0.0f;
            }
        }
#pragma unroll
        for (int q = 0; q < COUNT; ++q) {
            const T *v = reinterpret_cast<const T *>(&e[q]);
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (has[q]) low[q] = fmaf(to_f32(v[c]), x[q][c], low[q]);
        }
    }
}

// CTA: (8 / KS) runs of feature rows (32, or 16 gate rows with their 16 up rows) of one group times
// all of its tokens, 8 * NT at a time; KS warps share a run, each summing its part of K.
//
// With one token column set (NT = 1) two CTAs share an SM: 128 KB of weights in flight.
//
// Bound by memory, and for few groups by latency around it: 8 tokens of 8 of 64 experts, 2048 weight
// rows x 2048, gated, take 15.8 us for 67 MB (4.2 TB/s; 9.9 us at the measured bandwidth).
template <class T, class Y, int NT, bool GATED>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) few_rows_kernel(const GroupedArgs a, const int ks)
{
    extern __shared__ float parts[];  // kWarps x (8 NT) x kStride
    constexpr int kStride = kRowStride<2>;
    constexpr int kTokens = 8 * NT;
    constexpr int kFeat = GATED ? 16 : 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
    // a linear layer with adapters follows their inner products' kernel, which waited itself: only those
    // are waited for, below
    const bool adapted = !GATED && a.ad.b != nullptr;
    if (!adapted) chain_wait();
    else asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int group, first, rows;
    if (!nonempty_group(a, blockIdx.y, lane, group, first, rows)) return;
    const int block_feat = kWarps / ks * kFeat;
    const int64_t f0 = int64_t(blockIdx.x) * block_feat + warp / ks * kFeat;  // of this warp
    const T *W = static_cast<const T *>(a.W) + int64_t(group) * a.stridew;
    const T *w[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int64_t f = f0 + 8 * h + g + (GATED ? 0 : 16 * m);
            if (f >= a.N) f = a.N - 1;  // computed, not stored
            w[m][h] = W + (GATED && m == 1 ? f + a.N : f) * a.ldw;
        }
    const int64_t chunks = (a.K + 31) / 32, part = warp % ks;
    const int64_t kb = chunks * part / ks * 32;
    int64_t ke = chunks * (part + 1) / ks * 32;
    if (ke > a.K) ke = a.K;
    // unsigned: the last step may lead past 2^31
    for (unsigned n0 = blockIdx.z * kTokens; n0 < unsigned(rows); n0 += gridDim.z * kTokens) {
        const T *x[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const unsigned i = n0 + 8 * n + g;
            int64_t r = -1;
            if (i < unsigned(rows)) r = a.rows != nullptr ? __ldg(a.rows + first + i) : int64_t(first) + i;
            x[n] = r >= 0 && r < a.x_rows ? static_cast<const T *>(a.X) + r * a.ldx : nullptr;
        }
        float acc[2][NT][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[m][n][c] = 0.0f;
        warp_product<T, 2, NT>(w, x, kb, ke, a.K, lane, acc);
        __syncthreads();  // the partial tiles of the previous tokens have been read
        put_partial<2, NT>(parts + warp * kTokens * kStride, acc, lane);
        // adapters: their inner products come from the kernel before this one
        if (adapted) asm volatile("griddepcontrol.wait;" ::: "memory");
        __syncthreads();
        for (int i0 = threadIdx.x; i0 < block_feat * kTokens; i0 += NT * kThreads) {
            float low[NT];  // the adapters' part of the thread's next NT outputs
#pragma unroll
            for (int q = 0; q < NT; ++q) low[q] = 0.0f;
            if (adapted) {
                add_adapters<T, NT>(a, low, [&](int q, int64_t &p, int64_t &feat) {
                    const int i = i0 + q * kThreads, n = i / block_feat;
                    p = int64_t(first) + n0 + n;
                    feat = int64_t(blockIdx.x) * block_feat + i % block_feat;
                    return n < kTokens && n0 + n < unsigned(rows) && feat < a.N;
                });
            }
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                const int i = i0 + q * kThreads, f = i % block_feat, n = i / block_feat;
                const int64_t feat = int64_t(blockIdx.x) * block_feat + f;
                if (n >= kTokens || n0 + n >= unsigned(rows) || feat >= a.N) continue;
                const int64_t p = int64_t(first) + n0 + n;
                const float *src = parts + ((f / kFeat) * ks * kTokens + n) * kStride + f % kFeat;
                float v = 0.0f, u = 0.0f;
                for (int c = 0; c < ks; ++c) {
                    v += src[c * kTokens * kStride];
                    if (GATED) u += src[c * kTokens * kStride + 16];
                }
                if (GATED) {
                    if (a.pre != nullptr) {
                        T *pre = static_cast<T *>(a.pre) + p * a.ldp + feat;
                        pre[0] = from_f32<T>(v);
                        pre[a.N] = from_f32<T>(u);
                    }
                    v = v * sigmoid(v) * u;
                }
                static_cast<Y *>(a.Y)[p * a.ldy + feat] = from_f32<Y>(v + low[q]);
            }
        }
    }
    // a CTA without tokens of its own still orders this launch behind the one before it
    if (adapted) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// x = part 0 + part 1 + .. up to the last part's rounding.
template <class T, int PARTS> __device__ __forceinline__ void split(float x, uint16_t (&part)[PARTS])
{
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        const T a = from_f32<T>(x);
        const float f = to_f32(a);
        x = fabsf(f) < INFINITY ? x - f : 0.0f;  // an infinity is all in the first part
        part[i] = reinterpret_cast<const uint16_t &>(a);
    }
}

// Inner products of the adapters: inner[t][r] = scale * sum_k X[t][k] A_a[r][k] for 16 MT ranks of up to
// 8 NT tokens of one request, K split over the WARPS of the CTA.  Bound by latency for few tokens, where
// 16 warps share K; for a prompt by what the CTAs draw from L2, where one CTA takes 64 ranks, so that
// its tokens' rows are read once (launch_shrink_t's callers give the figures).  4096 tokens of 3
// requests, rank 64, K = 2048: 13 us, 51 MB drawn from L2.
//
// CTA i takes item i of an enumeration that needs no scan: cutting the tokens both at multiples of the
// tile and at the request boundaries, request s has the items t = segments[s] / tile + s ..
// segments[s + 1] / tile + s, so the request of item i is the last s whose first item is <= i.
//
// PARTS = 0 writes the few-rows form of the inner products, else the tcgen05 form (InnerLayout: the parts
// and the fp32 values), for which 8 NT is 32.
template <class T, int MT, int NT, int PARTS, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) shrink_kernel(const ShrinkArgs a)
{
    extern __shared__ float parts[];  // WARPS x (8 NT) x kStride
    constexpr int kThreads = 32 * WARPS, kTokens = 8 * NT, kStride = kRowStride<MT>;
    chain_wait();  // the product that follows may start on its weights and rows; it waits for inner
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
    auto seg = [&](int q) { return clamp_to(__ldg(a.segments + q), a.T); };
    if (PARTS == 0 && blockIdx.y == 0) {  // tokens of no request
        if (blockIdx.x == 0)
            for (int t = threadIdx.x; t < seg(0); t += kThreads) a.which[t] = -1;
        if (blockIdx.x == gridDim.x - 1)
            for (int t = seg(a.requests) + threadIdx.x; t < a.T; t += kThreads) a.which[t] = -1;
    }
    const int item = blockIdx.x;
    int lo = 0;  // last request whose first item is <= item, 32 candidates at a time
    for (int n = a.requests; n > 1;) {
        const int step = (n + 31) / 32, q = lo + lane * step;
        const bool before = lane * step < n && seg(q) / kTokens + q <= item;
        const int c = max(__popc(__ballot_sync(kFull, before)) - 1, 0);
        lo += c * step;
        n = min(step, n - c * step);
    }
    const int tile = item - lo;
    if (tile < 0) return;
    const int t0 = max(seg(lo), tile * kTokens);
    const int t1 = int(min(int64_t(seg(lo + 1)), int64_t(tile + 1) * kTokens));
    if (t0 >= t1) return;
    int ad = __ldg(a.adapters + lo);
    if (unsigned(ad) >= unsigned(a.n_adapters)) ad = -1;
    if (PARTS == 0 && blockIdx.y == 0)
        for (int t = t0 + int(threadIdx.x); t < t1; t += kThreads) a.which[t] = ad;
    if (ad < 0) return;

    const int r0 = blockIdx.y * 16 * MT;
    const T *A = static_cast<const T *>(a.A) + int64_t(ad) * a.stridea;
    const T *w[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) w[m][h] = A + int64_t(min(r0 + 16 * m + 8 * h + g, a.R - 1)) * a.lda;
    // tokens by their place in the tile, so that a tile is a block of the planes
    const T *x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t = tile * kTokens + 8 * n + g;
        x[n] = t >= t0 && t < t1 ? static_cast<const T *>(a.X) + int64_t(t) * a.ldx : nullptr;
    }
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[m][n][c] = 0.0f;
    const int64_t chunks = (a.K + 31) / 32;
    const int64_t kb = chunks * warp / WARPS * 32, ke = min(chunks * (warp + 1) / WARPS * 32, a.K);
    warp_product<T, MT, NT, WARPS == 16 ? 64 : 128>(w, x, kb, ke, a.K, lane, acc);
    put_partial<MT, NT>(parts + warp * kTokens * kStride, acc, lane);
    __syncthreads();
    const float scale = a.scales != nullptr ? __ldg(a.scales + ad) : 1.0f;
    const int ranks = min(16 * MT, a.R - r0);
    auto sum = [&](int n, int r) {  // of token n of the tile
        const float *src = parts + n * kStride + r;
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < WARPS; ++q) v += src[q * kTokens * kStride];
        return scale * v;
    };
    if constexpr (PARTS > 0) {
        static_assert(kTokens == 32, "blocks of 32 tokens");
        const InnerLayout in = inner_layout(a.T, a.requests, a.R, PARTS);
        float *values = reinterpret_cast<float *>(static_cast<char *>(a.planes) + in.values_at());
        uint16_t *plane = static_cast<uint16_t *>(a.planes) + int64_t(r0 / 64) * in.plane_rows * 64;
        const int64_t row0 = (int64_t(tile) + lo) * 32;
        for (int i = threadIdx.x; i < kTokens * 16 * MT; i += kThreads) {
            const int r = i % (16 * MT), n = i / (16 * MT), t = tile * kTokens + n;
            const bool there = r < ranks && t >= t0 && t < t1;
            const float v = there ? sum(n, r) : 0.0f;
            if (there) values[int64_t(t) * a.R + r0 + r] = v;
            uint16_t part[PARTS];
            split<T, PARTS>(v, part);
#pragma unroll
            for (int q = 0; q < PARTS; ++q)
                plane[int64_t(q) * in.blocks * in.plane_rows * 64 + (row0 + n) * 64 + r0 % 64 + r] = part[q];
        }
    } else {
        for (int i = threadIdx.x; i < ranks * (t1 - t0); i += kThreads) {
            const int r = i % ranks, t = t0 + i / ranks;
            a.inner[int64_t(t) * a.R + r0 + r] = sum(t - tile * kTokens, r);
        }
    }
}

template <class T, class Y, int NT, bool GATED>
cudaError_t launch_few_rows(const DeviceInfo &dev, const GroupedArgs &a, int64_t groups, int64_t depth, cudaStream_t stream)
{
    constexpr int kFeat = GATED ? 16 : 32;
    const int64_t runs = (a.N + kFeat - 1) / kFeat;
    // K is split as far as all warps still run at once, 16 to an SM, and a part is not below 256
    int ks = 1;
    while (ks < kWarps && 2 * groups * runs * depth * ks <= 16 * int64_t(dev.num_sms) && a.K / (2 * ks) >= 256) ks *= 2;
    const int64_t per = kWarps / ks;
    const size_t smem = size_t(kWarps) * 8 * NT * kRowStride<2> * sizeof(float);
    auto *kernel = few_rows_kernel<T, Y, NT, GATED>;
    const cudaError_t e = allow_smem_once(kernel, 100 * 1024);
    if (e != cudaSuccess) return e;
    const dim3 grid(unsigned((runs + per - 1) / per), unsigned(groups), unsigned(depth));
    return launch_chained(kernel, grid, kThreads, smem, 1, stream, a, ks);
}

template <class T, class Y> cudaError_t few_rows_t(const DeviceInfo &dev, const GroupedArgs &a, cudaStream_t stream)
{
    const int64_t groups = a.y_rows < a.groups ? a.y_rows : a.groups;  // at most that many have rows
    const int64_t mean = (a.y_rows + groups - 1) / groups;
    auto go = [&](auto nt) {
        constexpr int NT = decltype(nt)::value;
        // CTAs side by side for the tokens of the average group, at most 64
        int64_t depth = (mean + 8 * NT - 1) / (8 * NT);
        if (depth > 64) depth = 64;
        return a.gated ? launch_few_rows<T, Y, NT, true>(dev, a, groups, depth, stream)
                       : launch_few_rows<T, Y, NT, false>(dev, a, groups, depth, stream);
    };
    if (mean <= 8) return go(std::integral_constant<int, 1>{});
    if (mean <= 32) return go(std::integral_constant<int, 4>{});
    return go(std::integral_constant<int, 8>{});
}

template <class T, int MT, int NT, int PARTS, int WARPS> cudaError_t launch_shrink_t(const ShrinkArgs &a, cudaStream_t stream)
{
    constexpr size_t smem = size_t(WARPS) * 8 * NT * kRowStride<MT> * sizeof(float);
    auto *kernel = shrink_kernel<T, MT, NT, PARTS, WARPS>;
    const cudaError_t e = allow_smem_once(kernel, 100 * 1024);
    if (e != cudaSuccess) return e;
    static_assert(smem <= 100 * 1024, "dynamic shared memory");
    const dim3 grid(unsigned(a.T / (8 * NT) + a.requests), unsigned((a.R + 16 * MT - 1) / (16 * MT)));
    return launch_chained(kernel, grid, 32 * WARPS, smem, 1, stream, a);
}

// Ranks a CTA and warps, measured as whole calls (us).  Up to 16 ranks 16 warps: 4096 tokens of 3
// requests, 4096 x 4096, 91 against 100 with 8.  More ranks 8 warps with twice the registers: the same
// at rank 32 94 against 107, 300 tokens of 20 requests 27 against 29.  64 ranks a CTA where most
// requests fill a tile of 32 tokens: 8192 tokens of 7 requests, rank 64, 256 x 4096, 58 against 67, 512
// of 8 21 against 28, but 512 tokens of 64 requests 53 against 43 with 32 ranks.
template <class T, int NT, int PARTS> cudaError_t shrink_by_rank(const ShrinkArgs &a, cudaStream_t stream)
{
    if (a.R <= 16) return launch_shrink_t<T, 1, NT, PARTS, 16>(a, stream);
    if constexpr (PARTS == 0) return launch_shrink_t<T, 2, NT, PARTS, 16>(a, stream);
    else if (a.R > 32 && a.T >= 64 * int64_t(a.requests)) return launch_shrink_t<T, 4, NT, PARTS, 8>(a, stream);
    else return launch_shrink_t<T, 2, NT, PARTS, 8>(a, stream);
}

template <class T> cudaError_t shrink_t(const ShrinkArgs &a, cudaStream_t stream)
{
    if (a.inner == nullptr) {
        if (a.n_parts == 2) return shrink_by_rank<T, 4, 2>(a, stream);
        return shrink_by_rank<T, 4, 3>(a, stream);
    }
    // requests of one or a few tokens: 8 at a time (a 32-token tile would read its X rows in vain)
    return a.T <= 8 * int64_t(a.requests) ? shrink_by_rank<T, 1, 0>(a, stream) : shrink_by_rank<T, 4, 0>(a, stream);
}

}  // namespace

cudaError_t launch_few_rows(const DeviceInfo &dev, const GroupedArgs &a, cudaStream_t stream)
{
    if (a.type == GEMM_TYPE_F16)
        return a.y_type == GEMM_TYPE_F32 ? few_rows_t<__half, float>(dev, a, stream) : few_rows_t<__half, __half>(dev, a, stream);
    return a.y_type == GEMM_TYPE_F32 ? few_rows_t<__nv_bfloat16, float>(dev, a, stream)
                                     : few_rows_t<__nv_bfloat16, __nv_bfloat16>(dev, a, stream);
}

cudaError_t launch_shrink(const ShrinkArgs &a, cudaStream_t stream)
{
    return a.type == GEMM_TYPE_F16 ? shrink_t<__half>(a, stream) : shrink_t<__nv_bfloat16>(a, stream);
}

}  // namespace gemm
