// Routing to experts: scores, top-k within the kept groups, the plan that orders the slots by
// expert, and the gradient of the weights (semantics: include/gemm_gb300.h).
//
// One warp routes one token.  Lane l holds the experts v * 32 + l in registers, so a row of logits
// is read once in coalesced pieces; maxima, sums and the choice itself are warp reductions.  A
// choice compares 32-bit keys (the fp32 value with its bits mapped to unsigned order, 0 for an
// expert that is out), so one pick is two integer warp reductions: the largest key, then the lowest
// index that has it.  The kernel is bound by reading the logits for many tokens and by the launch
// for few.
//
// The plan is a stable counting sort of the slots by expert in one launch: one cluster of up to 8
// CTAs, every warp owning a contiguous run of slots and a histogram row of its own in shared
// memory.  Pass 1 counts (match.any gives the lanes of a warp that hold the same expert), the
// histograms are scanned over warps, CTAs (through distributed shared memory) and experts, pass 2
// places every slot at the running count of its warp.  No atomics, so the order never varies.  With
// few tokens the same launch routes them first (the warp's slots are then its own tokens').
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "routed_internal.h"

namespace cg = cooperative_groups;

namespace gemm {
namespace {

constexpr int kRouteWarps = 8;       // warps per CTA of the routing kernels
constexpr int kPlanWarps = 16;       // warps per CTA of the plan kernel
constexpr int kPlanMaxCluster = 8;   // portable cluster size
constexpr unsigned kFull = 0xffffffffu;

// Unsigned order of fp32 values; NaN and -inf (out of the choice) are 0, below every other value.
__device__ __forceinline__ uint32_t order_key(float v)
{
    if (!(v > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(v + 0.0f);  // -0 and +0 are one value
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

__device__ __forceinline__ float load_logit(int type, const void *p, int64_t i)
{
    if (type == GEMM_TYPE_F32) return static_cast<const float *>(p)[i];
    if (type == GEMM_TYPE_F16) return __half2float(static_cast<const __half *>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

// This lane's logits of row t with masks applied: -inf where masked, +inf as the largest finite
// value.
template <int V>
__device__ __forceinline__ void load_row(int type, const void *logits, int64_t ld, int64_t t, int E, int lane,
                                         float (&x)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * 32 + lane;
        float a = e < E ? load_logit(type, logits, t * ld + e) : -INFINITY;
        if (isnan(a)) a = -INFINITY;
        x[v] = fminf(a, FLT_MAX);
    }
}

// Scores of the row; 0 for masked logits.
template <int V>
__device__ __forceinline__ void scores(int score, const float (&x)[V], float (&s)[V])
{
    if (score == GEMM_SCORE_SIGMOID) {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = x[v] > -INFINITY ? sigmoid(x[v]) : 0.0f;
        return;
    }
    float m = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, x[v]);
    m = warp_max(m);
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        s[v] = x[v] > -INFINITY ? expf(x[v] - m) : 0.0f;
        sum += s[v];
    }
    sum = warp_sum(sum);
    if (sum > 0.0f) {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = s[v] / sum;
    }
}

// Routes token t with one warp.  `scratch`: E floats of shared memory of this warp.
template <int V>
__device__ void route_token(const RouteArgs &a, int64_t t, int lane, float *scratch)
{
    const int E = a.E;
    float x[V], s[V];
    load_row<V>(a.type, a.logits, a.ld, t, E, lane, x);
    scores<V>(a.score, x, s);
    uint32_t key[V];  // of the value the choice goes by
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * 32 + lane;
        float c = x[v];
        if (a.bias != nullptr && e < E && c > -INFINITY) c = s[v] + a.bias[e];
        key[v] = e < E ? order_key(c) : 0u;
    }
    if (a.groups > 1) {
        // Lane g takes run g: its group_top largest values.  The members are read from shared
        // memory starting at a different one in every lane, so that the lanes hit different banks.
        const int size = E / a.groups;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * 32 + lane;
            if (e < E) scratch[e] = key[v] == 0u ? -INFINITY : a.bias != nullptr ? s[v] + a.bias[e] : s[v];
        }
        __syncwarp();
        uint32_t gkey = 0u;
        if (lane < a.groups) {
            float b1 = -INFINITY, b2 = -INFINITY;
            int i = lane % size;
            for (int n = 0; n < size; ++n) {
                const float c = scratch[lane * size + i];
                b2 = fmaxf(b2, fminf(b1, c));
                b1 = fmaxf(b1, c);
                if (++i == size) i = 0;
            }
            gkey = order_key(a.group_top == 2 && b2 > -INFINITY ? b1 + b2 : b1);
        }
        uint32_t kept = 0u;
        for (int n = 0; n < a.groups_kept; ++n) {
            const uint32_t best = __reduce_max_sync(kFull, gkey);
            if (best == 0u) break;
            const int g = __ffs(__ballot_sync(kFull, gkey == best)) - 1;
            kept |= 1u << g;
            if (lane == g) gkey = 0u;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * 32 + lane;
            if (e < E && !((kept >> (e / size)) & 1u)) key[v] = 0u;
        }
        __syncwarp();  // scratch is read before the next token overwrites it
    }
    // Lane j keeps choice j.
    int my_id = -1;
    float my_s = 0.0f, sum = 0.0f;
    for (int j = 0; j < a.top_k; ++j) {
        uint32_t best = key[0];
        int at = 0;
#pragma unroll
        for (int v = 1; v < V; ++v)
            if (key[v] > best) {
                best = key[v];
                at = v;
            }
        const uint32_t top = __reduce_max_sync(kFull, best);
        if (top == 0u) break;
        const unsigned mine = best == top ? unsigned(at * 32 + lane) : 0xffffffffu;
        const int e = int(__reduce_min_sync(kFull, mine));
        float sv = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v * 32 + lane == e) {
                sv = s[v];
                key[v] = 0u;
            }
        sv = __shfl_sync(kFull, sv, e & 31);
        if (lane == j) {
            my_id = e;
            my_s = sv;
        }
        sum += sv;
    }
    if (lane < a.top_k) {
        float w = my_s;
        if (a.renormalise) w = sum > 0.0f ? my_s / sum : 0.0f;
        a.ids[t * a.top_k + lane] = my_id;
        a.weights[t * a.top_k + lane] = w * a.scale;
    }
}

template <int V>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const RouteArgs a)
{
    extern __shared__ float route_smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * kRouteWarps + warp;
    if (t < a.T) route_token<V>(a, t, lane, route_smem + warp * a.E);
}

// The plan (see the head of this file).  V > 0: the launch routes the tokens first.  Shared memory:
// kPlanWarps x E histogram rows, E totals of this CTA, E bases, and for V > 0 kPlanWarps x E floats.
template <int V>
__global__ void __launch_bounds__(kPlanWarps * 32) plan_kernel(const RouteArgs a)
{
    extern __shared__ uint32_t plan_smem[];
    const int E = a.E, k = a.top_k;
    uint32_t *hist = plan_smem, *total = hist + kPlanWarps * E, *base = total + E;
    __shared__ uint32_t warp_total[kPlanWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t warps = int64_t(ranks) * kPlanWarps, w = int64_t(rank) * kPlanWarps + warp;
    // this warp's tokens [t0, t1) and slots
    const int64_t t0 = a.T * w / warps, t1 = a.T * (w + 1) / warps;
    const int64_t s0 = t0 * k, s1 = t1 * k;

    for (int i = threadIdx.x; i < kPlanWarps * E; i += blockDim.x) hist[i] = 0u;
    if constexpr (V > 0) {
        float *scratch = reinterpret_cast<float *>(base + E) + warp * E;
        for (int64_t t = t0; t < t1; ++t) route_token<V>(a, t, lane, scratch);
    }
    __syncthreads();

    uint32_t *mine = hist + warp * E;
    auto expert_of = [&](int64_t s) {
        const int e = s < s1 ? a.ids[s] : -1;
        return e >= 0 && e < E ? e : -1;
    };
    // slots 4 x 32 at a time, so that four loads are in flight
    for (int64_t s = s0; s < s1; s += 128) {
        int e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = expert_of(s + 32 * i + lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned same = __match_any_sync(kFull, e[i]);
            if (e[i] >= 0 && lane == __ffs(same) - 1) mine[e[i]] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        uint32_t run = 0;
#pragma unroll
        for (int i = 0; i < kPlanWarps; ++i) {
            const uint32_t n = hist[i * E + e];
            hist[i * E + e] = run;
            run += n;
        }
        total[e] = run;
    }
    cluster.sync();
    // Exclusive scan of the experts' totals over the cluster; thread i holds experts 2 i, 2 i + 1.
    uint32_t all[2] = {0, 0}, before[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = 2 * threadIdx.x + i;
        if (e < E)
            for (int r = 0; r < ranks; ++r) {
                const uint32_t n = cluster.map_shared_rank(total, r)[e];
                if (r < rank) before[i] += n;
                all[i] += n;
            }
    }
    uint32_t incl = all[0] + all[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t n = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += n;
    }
    if (lane == 31) warp_total[warp] = incl;
    __syncthreads();
    uint32_t first = incl - all[0] - all[1];
    for (int i = 0; i < warp; ++i) first += warp_total[i];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = 2 * threadIdx.x + i;
        if (e < E) {
            base[e] = first + before[i];
            if (rank == 0) {
                a.offsets[e] = int32_t(first);
                if (e == E - 1) a.offsets[E] = int32_t(first + all[i]);
            }
        }
        first += all[i];
    }
    __syncthreads();
    for (int64_t s = s0; s < s1; s += 128) {
        int e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = expert_of(s + 32 * i + lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t slot = s + 32 * i + lane;
            const unsigned same = __match_any_sync(kFull, e[i]);
            if (e[i] >= 0) {
                const uint32_t p = base[e[i]] + mine[e[i]] + __popc(same & ((1u << lane) - 1u));
                a.where[slot] = int32_t(p);
                a.tokens[p] = int32_t(slot / k);
            } else if (slot < s1) {
                a.where[slot] = -1;
            }
            __syncwarp();
            if (e[i] >= 0 && lane == __ffs(same) - 1) mine[e[i]] += __popc(same);
            __syncwarp();
        }
    }
    cluster.sync();  // no CTA leaves while another may still read its totals
}

template <int V>
__global__ void __launch_bounds__(kRouteWarps * 32)
route_backward_kernel(const RouteArgs a, const float *dweights, const int32_t *ids, void *dlogits, int64_t ldd)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * kRouteWarps + warp;
    if (t >= a.T) return;
    const int E = a.E, k = a.top_k;
    float x[V], s[V], ds[V];
    load_row<V>(a.type, a.logits, a.ld, t, E, lane, x);
    scores<V>(a.score, x, s);
#pragma unroll
    for (int v = 0; v < V; ++v) ds[v] = 0.0f;
    // lane j holds choice j: its expert, score and gradient
    int id = -1;
    float dw = 0.0f, sel = 0.0f;
    if (lane < k) {
        id = ids[t * k + lane];
        if (id < 0 || id >= E) id = -1;
        if (id >= 0) dw = dweights[t * k + lane];
    }
    for (int j = 0; j < k; ++j) {
        const int e = __shfl_sync(kFull, id, j);
        float sv = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v * 32 + lane == e) sv = s[v];
        sv = __shfl_sync(kFull, sv, e & 31);
        if (lane == j && id >= 0) sel = sv;
    }
    float g = a.scale * dw;
    if (a.renormalise) {
        const float S = warp_sum(sel);
        const float p = S > 0.0f ? sel / S : 0.0f;
        const float mean = warp_sum(dw * p);
        g = S > 0.0f ? a.scale * (dw - mean) / S : 0.0f;
    }
    for (int j = 0; j < k; ++j) {
        const int e = __shfl_sync(kFull, id, j);
        const float gj = __shfl_sync(kFull, g, j);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v * 32 + lane == e) ds[v] += gj;
    }
    float mean = 0.0f;  // sum of ds * s; 0 by its definition when the weights are renormalised
    if (a.score == GEMM_SCORE_SOFTMAX && !a.renormalise) {
#pragma unroll
        for (int v = 0; v < V; ++v) mean += ds[v] * s[v];
        mean = warp_sum(mean);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * 32 + lane;
        if (e >= E) continue;
        // a masked logit has score 0 and so gradient 0
        float d = a.score == GEMM_SCORE_SOFTMAX ? s[v] * (ds[v] - mean) : ds[v] * s[v] * (1.0f - s[v]);
        if (!(x[v] > -INFINITY)) d = 0.0f;
        const int64_t i = t * ldd + e;
        if (a.type == GEMM_TYPE_F32) static_cast<float *>(dlogits)[i] = d;
        else if (a.type == GEMM_TYPE_F16) static_cast<__half *>(dlogits)[i] = __float2half_rn(d);
        else static_cast<__nv_bfloat16 *>(dlogits)[i] = __float2bfloat16_rn(d);
    }
}

template <int V>
cudaError_t launch_plan_t(const RouteArgs &a, cudaStream_t stream)
{
    const size_t smem = (size_t(kPlanWarps) + 2 + (V > 0 ? kPlanWarps : 0)) * size_t(a.E) * 4;
    cudaError_t e = allow_smem_once(plan_kernel<V>, 140 * 1024);
    if (e != cudaSuccess) return e;
    // CTAs enough that a warp has at most a few tokens to route, or 1024 slots to sort; a power of 2
    const int64_t per_cta = V > 0 ? 2 * kPlanWarps : 1024;
    int ranks = 1;
    while (ranks < kPlanMaxCluster && a.T * (V > 0 ? 1 : a.top_k) > ranks * per_cta) ranks *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ranks);
    cfg.blockDim = dim3(kPlanWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ranks;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, plan_kernel<V>, a);
    if (e == cudaSuccess) count_launches();
    return e;
}

template <class F>
cudaError_t by_values_per_lane(int E, F f)
{
    if (E <= 32) return f(std::integral_constant<int, 1>{});
    if (E <= 64) return f(std::integral_constant<int, 2>{});
    if (E <= 128) return f(std::integral_constant<int, 4>{});
    if (E <= 256) return f(std::integral_constant<int, 8>{});
    if (E <= 512) return f(std::integral_constant<int, 16>{});
    return f(std::integral_constant<int, 32>{});
}

}  // namespace

// Few tokens: one launch routes and plans (the routing then runs on the plan's 8 CTAs only, so
// only up to kFusedTokens tokens, and E <= 256 so that two E-sized shared rows per warp fit).
constexpr int64_t kFusedTokens = 512;

cudaError_t launch_plan(int64_t T, int E, int top_k, const int32_t *ids, int32_t *offsets, int32_t *tokens,
                        int32_t *where, cudaStream_t stream)
{
    RouteArgs a{};
    a.T = T;
    a.E = E;
    a.top_k = top_k;
    a.ids = const_cast<int32_t *>(ids);
    a.offsets = offsets;
    a.tokens = tokens;
    a.where = where;
    return launch_plan_t<0>(a, stream);
}

cudaError_t launch_route(const RouteArgs &a, cudaStream_t stream)
{
    const bool plan = a.offsets != nullptr;
    if (plan && (a.T == 0 || (a.T <= kFusedTokens && a.E <= 256))) {
        if (a.T == 0) return launch_plan(0, a.E, a.top_k, a.ids, a.offsets, a.tokens, a.where, stream);
        if (a.E <= 32) return launch_plan_t<1>(a, stream);
        if (a.E <= 64) return launch_plan_t<2>(a, stream);
        if (a.E <= 128) return launch_plan_t<4>(a, stream);
        return launch_plan_t<8>(a, stream);
    }
    if (a.T == 0) return cudaSuccess;
    const cudaError_t e = by_values_per_lane(a.E, [&](auto v) {
        const unsigned blocks = unsigned((a.T + kRouteWarps - 1) / kRouteWarps);
        route_kernel<decltype(v)::value><<<blocks, kRouteWarps * 32, size_t(kRouteWarps) * a.E * 4, stream>>>(a);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    count_launches();
    return plan ? launch_plan(a.T, a.E, a.top_k, a.ids, a.offsets, a.tokens, a.where, stream) : cudaSuccess;
}

cudaError_t launch_route_backward(const RouteArgs &a, const float *dweights, const int32_t *ids, void *dlogits,
                                  int64_t ldd, cudaStream_t stream)
{
    const cudaError_t e = by_values_per_lane(a.E, [&](auto v) {
        const unsigned blocks = unsigned((a.T + kRouteWarps - 1) / kRouteWarps);
        route_backward_kernel<decltype(v)::value>
            <<<blocks, kRouteWarps * 32, 0, stream>>>(a, dweights, ids, dlogits, ldd);
        return cudaGetLastError();
    });
    if (e == cudaSuccess) count_launches();
    return e;
}

}  // namespace gemm
