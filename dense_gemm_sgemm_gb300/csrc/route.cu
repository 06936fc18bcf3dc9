// Routing to experts: scores, top-k within the kept groups, the plan that orders the slots by
// expert, and the gradient of the weights (semantics: include/gemm_gb300.h).
//
// One warp routes one token.  Lane l holds the experts V l .. V l + V - 1 in registers, read with
// 16-byte loads where the row allows it; maxima, sums and the choice itself are warp reductions.  A
// choice compares 32-bit keys (the fp32 value with its bits mapped to unsigned order, 0 for an expert
// that is out), so one pick is one integer warp maximum and a ballot, whose lowest lane holds the
// lowest index.  Runs of experts that are whole lanes, a power of two of them, are reduced by
// shuffles, others through shared memory.  Bound by instructions: 16384 tokens of 256 experts, sigmoid,
// bias, 8 in 4 of 8 runs, take 21 us (25 alone and from cold caches) at 72% of the issue slots, 1370
// instructions a token, a third of them in the eight picks.
//
// The plan is a stable counting sort of the slots by expert in one launch: one cluster of CTAs, every
// warp owning a contiguous run of slots and a histogram row of its own in shared memory.  Pass 1
// counts (match.any gives the lanes of a warp that hold the same expert) and keeps each slot's rank
// in its warp; the histograms are scanned over warps, CTAs (through distributed shared
// memory) and experts; pass 2 adds them.  No atomics, so the order never varies.  Bound by latency on
// 16 SMs: 131072 slots of 256 experts take 17.4 us (21 alone and from cold caches).  With few tokens the
// same launch routes them first (the warp's slots are then its own tokens').
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "routed_internal.h"

namespace cg = cooperative_groups;

namespace gemm {
namespace {

constexpr int kRouteWarps = 8;  // warps per CTA of the routing kernels
// Warps per CTA of the plan kernel and CTAs of its cluster.  The form that routes as well needs the
// registers of 16 warps; the other takes all it can get (16 CTAs of 32 warps; 8 of 16 measured 38 us
// on 131072 slots, see launch_plan_t).
template <int V> constexpr int plan_warps = V > 0 ? 16 : 32;
template <int V> constexpr int plan_cluster = V > 0 ? 8 : 16;
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

// Elements of this lane of row t.  `wide`: rows start on 16-byte boundaries.
template <class T, int V>
__device__ __forceinline__ void load_lane(const T *row, int E, int lane, bool wide, float (&x)[V])
{
    constexpr int kPiece = 16 / sizeof(T) < V ? 16 / sizeof(T) : V;
    if (wide && lane * V + V <= E && kPiece * sizeof(T) == 16) {
#pragma unroll
        for (int v = 0; v < V; v += kPiece) {
            const uint4 q = load_now(reinterpret_cast<const uint4 *>(row + lane * V + v));
#pragma unroll
            for (int i = 0; i < kPiece; ++i) x[v + i] = to_f32(reinterpret_cast<const T *>(&q)[i]);
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = lane * V + v < E ? to_f32(row[lane * V + v]) : -INFINITY;
    }
}

template <class T, int V>
__device__ __forceinline__ void store_lane(T *row, int E, int lane, bool wide, const float (&x)[V])
{
    constexpr int kPiece = 16 / sizeof(T) < V ? 16 / sizeof(T) : V;
    if (wide && lane * V + V <= E && kPiece * sizeof(T) == 16) {
#pragma unroll
        for (int v = 0; v < V; v += kPiece) {
            uint4 q;
#pragma unroll
            for (int i = 0; i < kPiece; ++i) reinterpret_cast<T *>(&q)[i] = from_f32<T>(x[v + i]);
            *reinterpret_cast<uint4 *>(row + lane * V + v) = q;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane * V + v < E) row[lane * V + v] = from_f32<T>(x[v]);
    }
}

// This lane's logits of row t with masks applied: -inf where masked, +inf as the largest finite
// value.
template <int V>
__device__ __forceinline__ void load_row(const RouteArgs &a, int64_t t, int lane, float (&x)[V])
{
    if (a.type == GEMM_TYPE_F32)
        load_lane<float, V>(static_cast<const float *>(a.logits) + t * a.ld, a.E, lane, a.wide, x);
    else if (a.type == GEMM_TYPE_F16)
        load_lane<__half, V>(static_cast<const __half *>(a.logits) + t * a.ld, a.E, lane, a.wide, x);
    else
        load_lane<__nv_bfloat16, V>(static_cast<const __nv_bfloat16 *>(a.logits) + t * a.ld, a.E, lane, a.wide, x);
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = isnan(x[v]) ? -INFINITY : fminf(x[v], FLT_MAX);
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

// Keys of the runs, on the first lane of each (`lanes` lanes a run) or on lane g for run g.
template <int V>
__device__ __forceinline__ uint32_t run_keys(const RouteArgs &a, const float (&value)[V], int lane, int lanes, float *scratch)
{
    float b1 = -INFINITY, b2 = -INFINITY;
    if (lanes > 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            b2 = fmaxf(b2, fminf(b1, value[v]));
            b1 = fmaxf(b1, value[v]);
        }
        for (int o = 1; o < lanes; o <<= 1) {
            const float c1 = __shfl_xor_sync(kFull, b1, o), c2 = __shfl_xor_sync(kFull, b2, o);
            b2 = fmaxf(fminf(b1, c1), fmaxf(b2, c2));
            b1 = fmaxf(b1, c1);
        }
        if (lane % lanes != 0) b1 = -INFINITY;
    } else {
        // Lane g takes run g.  The members are read starting at a different one in every lane, so
        // that the lanes hit different banks.
        const int size = a.E / a.groups;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane * V + v < a.E) scratch[lane * V + v] = value[v];
        __syncwarp();
        if (lane < a.groups) {
            int i = lane % size;
            for (int n = 0; n < size; ++n) {
                const float c = scratch[lane * size + i];
                b2 = fmaxf(b2, fminf(b1, c));
                b1 = fmaxf(b1, c);
                if (++i == size) i = 0;
            }
        }
        __syncwarp();  // scratch is read before the next token overwrites it
    }
    return order_key(a.group_top == 2 && b2 > -INFINITY ? b1 + b2 : b1);
}

// Routes token t with one warp.  `scratch`: E floats of shared memory of this warp.
template <int V>
__device__ void route_token(const RouteArgs &a, int64_t t, int lane, float *scratch)
{
    const int E = a.E;
    float x[V], s[V];
    load_row<V>(a, t, lane, x);
    scores<V>(a.score, x, s);
    // what a run's value is made of, and the key of what the choice goes by
    float value[V];
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane * V + v;
        const bool live = e < E && x[v] > -INFINITY;
        value[v] = !live ? -INFINITY : a.bias != nullptr ? s[v] + load_now(a.bias + e) : s[v];
        if (isnan(value[v])) value[v] = -INFINITY;
        key[v] = order_key(a.bias != nullptr ? value[v] : live ? x[v] : -INFINITY);
    }
    if (a.groups > 1) {
        const int size = E / a.groups;
        // whole lanes a run, a power of two of them: reduced by shuffles
        const int lanes = size % V == 0 && ((size / V) & (size / V - 1)) == 0 ? size / V : 0;
        uint32_t gkey = run_keys<V>(a, value, lane, lanes, scratch);
        uint32_t kept = 0u;  // bit of the lane that holds the run's key
        for (int n = 0; n < a.groups_kept; ++n) {
            const uint32_t best = __reduce_max_sync(kFull, gkey);
            if (best == 0u) break;
            const int at = __ffs(__ballot_sync(kFull, gkey == best)) - 1;
            kept |= 1u << at;
            if (lane == at) gkey = 0u;
        }
        if (lanes > 0) {
            if (!((kept >> (lane & ~(lanes - 1))) & 1u)) {
#pragma unroll
                for (int v = 0; v < V; ++v) key[v] = 0u;
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = lane * V + v;
                if (e < E && !((kept >> (e / size)) & 1u)) key[v] = 0u;
            }
        }
    }
    // Lane j keeps choice j; its score comes from shared memory in the end.
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (lane * V + v < E) scratch[lane * V + v] = s[v];
    int my_id = -1;
    for (int j = 0; j < a.top_k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) best = max(best, key[v]);
        const uint32_t top = __reduce_max_sync(kFull, best);
        if (top == 0u) break;
        const int owner = __ffs(__ballot_sync(kFull, best == top)) - 1;
        int at = 0;
        if (lane == owner) {
#pragma unroll
            for (int v = V - 1; v >= 0; --v)  // the lowest of equals
                if (key[v] == top) at = v;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v == at) key[v] = 0u;
        }
        const int e = __shfl_sync(kFull, owner * V + at, owner);
        if (lane == j) my_id = e;
    }
    __syncwarp();
    const float my_s = my_id >= 0 ? scratch[my_id] : 0.0f;
    const float sum = warp_sum(my_s);
    __syncwarp();  // scratch is read before the next token overwrites it
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
    chain_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * kRouteWarps + warp;
    if (t < a.T) route_token<V>(a, t, lane, route_smem + warp * a.E);
}

// The plan (see the head of this file).  V > 0: the launch routes the tokens first.  Shared memory,
// with W warps: W x E histogram rows, E totals of this CTA, E bases, and for V > 0 W x E floats.
template <int V>
__global__ void __launch_bounds__(32 * plan_warps<V>) plan_kernel(const RouteArgs a)
{
    extern __shared__ uint32_t plan_smem[];
    constexpr int kWarps = plan_warps<V>;
    const int E = a.E, k = a.top_k;
    uint32_t *hist = plan_smem, *total = hist + kWarps * E, *base = total + E;
    __shared__ uint32_t warp_total[kWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t warps = int64_t(ranks) * kWarps, w = int64_t(rank) * kWarps + warp;
    // this warp's tokens [t0, t1) and slots (below 2^31 of them: 32-bit divisions)
    const int64_t t0 = a.T * w / warps, t1 = a.T * (w + 1) / warps;
    const unsigned s0 = unsigned(t0 * k), s1 = unsigned(t1 * k);

    for (int i = threadIdx.x; i < kWarps * E; i += blockDim.x) hist[i] = 0u;
    chain_wait();
    if constexpr (V > 0) {
        float *scratch = reinterpret_cast<float *>(base + E) + warp * E;
        for (int64_t t = t0; t < t1; ++t) route_token<V>(a, t, lane, scratch);
    }
    __syncthreads();

    uint32_t *mine = hist + warp * E;
    // Slots 8 x 32 at a time, so that their loads are in flight together.  The first 256 slots of a warp
    // keep their experts and ranks in registers, the others leave their ranks in `where`.
    int held[8], held_rank[8];
    auto count = [&](unsigned s, int (&e)[8], int (&rank_in_warp)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const unsigned slot = s + 32 * i + lane;
            e[i] = slot < s1 ? a.ids[slot] : -1;
            if (e[i] < 0 || e[i] >= E) e[i] = -1;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            rank_in_warp[i] = -1;
            if (s + 32 * i >= s1) continue;  // the same for the warp
            const unsigned same = __match_any_sync(kFull, e[i]);
            const uint32_t before = e[i] >= 0 ? mine[e[i]] : 0u;
            __syncwarp();
            if (e[i] >= 0 && lane == __ffs(same) - 1) mine[e[i]] = before + __popc(same);
            __syncwarp();
            if (e[i] >= 0) rank_in_warp[i] = int(before + __popc(same & ((1u << lane) - 1u)));
        }
    };
    count(s0, held, held_rank);
    for (unsigned s = s0 + 256; s < s1; s += 256) {
        int e[8], rank_in_warp[8];
        count(s, e, rank_in_warp);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (s + 32 * i + lane < s1) a.where[s + 32 * i + lane] = rank_in_warp[i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        uint32_t run = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
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
        if (e < E) {
            uint32_t n[plan_cluster<V>];  // all of the remote reads in flight together
#pragma unroll
            for (int r = 0; r < plan_cluster<V>; ++r) n[r] = r < ranks ? cluster.map_shared_rank(total, r)[e] : 0u;
#pragma unroll
            for (int r = 0; r < plan_cluster<V>; ++r) {
                if (r < rank) before[i] += n[r];
                all[i] += n[r];
            }
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
    // the totals have been read: no CTA leaves before all have come here (waited for below)
    if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    auto put = [&](unsigned slot, int e, int rank_in_warp) {
        if (rank_in_warp >= 0) {
            const uint32_t p = base[e] + mine[e] + uint32_t(rank_in_warp);
            a.where[slot] = int32_t(p);
            a.tokens[p] = int32_t(slot / unsigned(k));
        } else {
            a.where[slot] = -1;
        }
    };
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (s0 + 32 * i + lane < s1) put(s0 + 32 * i + lane, held[i], held_rank[i]);
    for (unsigned s = s0 + 256; s < s1; s += 256) {
        int e[8], rank_in_warp[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // the ranks that this very thread wrote above
            const unsigned slot = s + 32 * i + lane;
            rank_in_warp[i] = slot < s1 ? a.where[slot] : -1;
            e[i] = slot < s1 ? a.ids[slot] : 0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (s + 32 * i + lane < s1) put(s + 32 * i + lane, e[i], rank_in_warp[i]);
    }
    if (ranks > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// Gradient of the weights w_j = scale * s_j (/ S, the sum of the chosen scores, when renormalised) for
// one token a warp: ds_j = scale * dw_j, or scale * (dw_j - sum_i dw_i s_i / S) / S; then
// dx_e = s_e (ds_e - sum ds s) for softmax, ds_e s_e (1 - s_e) for sigmoid.  When renormalised the factors
// s_e and 1 / S enter as the ordinary s_e / S, since 1 / S overflows where all of the chosen scores are tiny
// (a bias chooses such experts), and sum ds s is 0 by its definition.  Lane j takes choice j and
// puts its gradient by expert into shared memory, so that every lane stores its own experts in wide
// pieces.  Bound by the launch and the latency of one row: 8191 tokens of 128 experts, top 6, 5.0 us.
template <int V>
__global__ void __launch_bounds__(kRouteWarps * 32)
route_backward_kernel(const RouteArgs a, const float *dweights, const int32_t *ids, void *dlogits, int64_t ldd, bool wide)
{
    chain_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * kRouteWarps + warp;
    if (t >= a.T) return;
    const int E = a.E, k = a.top_k;
    extern __shared__ float route_smem[];
    float *row = route_smem + warp * E;  // by expert: scores, then gradients of scores
    float x[V], s[V], ds[V];
    load_row<V>(a, t, lane, x);
    scores<V>(a.score, x, s);
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (lane * V + v < E) row[lane * V + v] = s[v];
    __syncwarp();
    // lane j holds choice j: its expert, score and gradient (renormalised: with the factor s)
    int id = -1;
    float dw = 0.0f, sel = 0.0f;
    if (lane < k) {
        id = ids[t * k + lane];
        if (id < 0 || id >= E) id = -1;
        if (id >= 0) {
            dw = dweights[t * k + lane];
            sel = row[id];
        }
    }
    float g = a.scale * dw;
    if (a.renormalise) {
        const float S = warp_sum(sel);
        const float p = S > 0.0f ? sel / S : 0.0f;
        const float mean = warp_sum(dw * p);
        g = a.scale * (dw - mean) * p;  // times s already
    }
    __syncwarp();
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (lane * V + v < E) row[lane * V + v] = 0.0f;
    __syncwarp();
    // an expert named twice gets the sum, in the order of the choices
    const unsigned same = __match_any_sync(kFull, id);
    if (__any_sync(kFull, id >= 0 && (same & (same - 1u)) != 0u)) {
        float all = 0.0f;
        for (int j = 0; j < k; ++j) {
            const float gj = __shfl_sync(kFull, g, j);
            if ((same >> j) & 1u) all += gj;
        }
        g = all;
    }
    if (id >= 0 && lane == __ffs(same) - 1) row[id] = g;
    __syncwarp();
#pragma unroll
    for (int v = 0; v < V; ++v) ds[v] = lane * V + v < E ? row[lane * V + v] : 0.0f;
    float mean = 0.0f;  // sum of ds * s
    if (a.score == GEMM_SCORE_SOFTMAX && !a.renormalise) {
#pragma unroll
        for (int v = 0; v < V; ++v) mean += ds[v] * s[v];
        mean = warp_sum(mean);
    }
    float d[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        // a masked logit has score 0 and so gradient 0
        if (a.score == GEMM_SCORE_SOFTMAX) d[v] = a.renormalise ? ds[v] : s[v] * (ds[v] - mean);
        else d[v] = (a.renormalise ? ds[v] : ds[v] * s[v]) * (1.0f - s[v]);
        if (!(x[v] > -INFINITY)) d[v] = 0.0f;
    }
    if (a.type == GEMM_TYPE_F32) store_lane<float, V>(static_cast<float *>(dlogits) + t * ldd, E, lane, wide, d);
    else if (a.type == GEMM_TYPE_F16) store_lane<__half, V>(static_cast<__half *>(dlogits) + t * ldd, E, lane, wide, d);
    else store_lane<__nv_bfloat16, V>(static_cast<__nv_bfloat16 *>(dlogits) + t * ldd, E, lane, wide, d);
}

template <int V>
cudaError_t launch_plan_t(const RouteArgs &a, cudaStream_t stream)
{
    constexpr int kWarps = plan_warps<V>;
    const size_t smem = (size_t(kWarps) + 2 + (V > 0 ? kWarps : 0)) * size_t(a.E) * 4;
    cudaError_t e = allow_smem_once(plan_kernel<V>, 140 * 1024);
    if (e != cudaSuccess) return e;
    // CTAs enough that a warp has at most a few tokens to route, or 256 slots to sort at once; a
    // power of 2
    const int64_t per_cta = V > 0 ? 2 * kWarps : 128 * kWarps;
    int ranks = 1;
    while (ranks < plan_cluster<V> && a.T * (V > 0 ? 1 : a.top_k) > ranks * per_cta) ranks *= 2;
    if (ranks > 8 && allow_large_cluster_once(plan_kernel<V>) != cudaSuccess) {
        cudaGetLastError();
        ranks = 8;
    }
    return launch_chained(plan_kernel<V>, dim3(ranks), kWarps * 32, smem, ranks, stream, a);
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

static bool wide_rows(int type, const void *p, int64_t ld)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % (type == GEMM_TYPE_F32 ? 4 : 8) == 0;
}

// Few tokens: one launch routes and plans (the routing then runs on the plan's 8 CTAs only, so
// only up to kFusedTokens tokens, and for E <= 256: more experts would fit its shared memory, but want two
// more instances of the kernel for calls that have not been measured).
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

cudaError_t launch_route(const RouteArgs &call, cudaStream_t stream)
{
    RouteArgs a = call;
    a.wide = wide_rows(a.type, a.logits, a.ld);
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
        return launch_chained(route_kernel<decltype(v)::value>, dim3(blocks), kRouteWarps * 32,
                              size_t(kRouteWarps) * a.E * 4, 1, stream, a);
    });
    if (e != cudaSuccess) return e;
    return plan ? launch_plan_t<0>(a, stream) : cudaSuccess;
}

cudaError_t launch_route_backward(const RouteArgs &call, const float *dweights, const int32_t *ids, void *dlogits,
                                  int64_t ldd, cudaStream_t stream)
{
    RouteArgs a = call;
    a.wide = wide_rows(a.type, a.logits, a.ld);
    const bool wide = wide_rows(a.type, dlogits, ldd);
    return by_values_per_lane(a.E, [&](auto v) {
        const unsigned blocks = unsigned((a.T + kRouteWarps - 1) / kRouteWarps);
        return launch_chained(route_backward_kernel<decltype(v)::value>, dim3(blocks), kRouteWarps * 32,
                              size_t(kRouteWarps) * a.E * 4, 1, stream, a, dweights, ids, dlogits, ldd, wide);
    });
}

}  // namespace gemm
