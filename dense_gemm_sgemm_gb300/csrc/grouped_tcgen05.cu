// Grouped products with many rows per weight matrix on the tcgen05 tensor cores: the grouped linear
// layer (either storage of W, gated or not), the linear layer with adapters, and the weight gradient
// (semantics: include/gemm_gb300.h).
//
// Forward and input gradient.  A group's rows are many or few and never a multiple of a tile, so the
// features take the MMA's m side, where tiles are fixed, and the tokens its n side, which is any
// multiple of 32 up to 256: D[feature][token] = W_g X^T.  Two CTAs on neighbouring SMs form a 256 x n
// tile (tcgen05.mma.cta_group::2; each loads its own 128 weight rows and half of the tokens).  Warps:
//   0     TMA producer of the weights, per 64-wide K slice;
//   10    TMA producer of the token rows: contiguous rows in boxes of 128, 64, 32 and 16, gathered
//         rows four at a time (tile::gather4) by all lanes;
//   1     MMA issuer (of the pair's first CTA) and TMEM owner, two 256-column accumulators;
//   2-9   epilogue: one TMEM lane is one feature, so 32 tokens x 32 features pass through shared
//         memory per warp and leave by TMA stores, those of a group's last tokens as 16-byte pieces
//         of its rows.
// gated: a CTA's 128 rows are 64 gate rows and their 64 up rows; the warps that hold a gate and its
// up exchange halves through shared memory.  Adapters: behind a tile's last K slice come the slices
// of its requests' low-rank products, B_a on the m side and the inner products on the n side, over the
// columns of the request only (see TileRequests); the kernel ahead computes the inner products in
// 16-bit parts that sum to them (launch_shrink).  On the CUDA cores of the epilogue this product was
// bound by broadcasting the inner products from shared memory (8192 tokens, rank 64, 4096 x 4096, whole
// calls: 369 us, as slices 226 at first), with mma.sync there by tcgen05, which goes first (371 us).  An
// infinity or NaN in an adapter's B would spoil the columns of its neighbours, where it meets zeros: the
// epilogue notes the tiles whose sums are not finite, and the pair computes those a second time with such
// adapters' products in fp32 on the CUDA cores, as well as those whose inner products the 16-bit parts
// cannot hold (TileRequests).
//
// Weight gradient.  dW_g[n][k] sums over the group's positions, the K dimension of this product,
// both operands "transposed" (MN-major).  Slices are 64 positions; the last one of a group also holds
// rows of the next group, which a cleaner warp overwrites with zeros in shared memory before the MMAs
// read them (multiplying them by zero would let their infinities through).
//
// Every wait is bounded: when one expires the kernel raises the device's error word, stops all
// roles, waits (bounded) for its own copies and MMAs in flight, frees its TMEM and returns.
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdlib>
#include <cstring>

#include "routed_internal.h"
#include "tcgen05_ptx.cuh"
#include "tcgen05_roles.cuh"
#include "tensor_map.h"

namespace gemm {
namespace {

constexpr int kStageA = 128 * 128;     // bytes: 128 weight rows (or 64 k rows x 2 boxes) of 128 bytes
constexpr int kMaxStageB = 128 * 128;  // bytes: up to 128 token rows
constexpr int kRingBytes = 5 * (kStageA + kMaxStageB);
constexpr int kMaxStages = 9;  // of the smallest stage: 16 token rows, 18 KB
constexpr int kEpiWarps = 8;  // two for every 32 TMEM lanes, taking the columns in turn
constexpr int kEpiBytes = kEpiWarps * 32 * 32 * 4;  // a 32 x 32 fp32 staging tile each
constexpr int kBarBytes = 512;
constexpr int kTmemCols = 512, kAccCols = 256;
constexpr int kMaxGroups = 1024;
constexpr int kTableBytes = 2 * (kMaxGroups + 2) * 4;  // first position and first unit of every group
constexpr int kSmemBytes = kRingBytes + kEpiBytes + kBarBytes + kTableBytes + 1024;
static_assert(kSmemBytes <= 227 * 1024, "one CTA per SM");
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ int clamp_to(int v, int64_t hi) { return v < 0 ? 0 : v > hi ? int(hi) : v; }

// ------------------------------------------------------------------ shared pieces
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t c0, int32_t c1)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
// Columns from c0 of four rows (one-row boxes); a row outside the tensor arrives as zeros.
__device__ __forceinline__ void tma_gather4_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t c0, int4 r)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w)
        : "memory");
}

// The ring: as many stages of kStageA + b_bytes as fit, for the bytes in flight that small tiles are
// short of (128 groups of 4 rows, 2048 x 2048: 158 us, with five stages 167).
__host__ __device__ constexpr int ring_stages(int b_bytes)
{
    return kRingBytes / (kStageA + b_bytes) < kMaxStages ? kRingBytes / (kStageA + b_bytes) : kMaxStages;
}

// Barriers and the rest of shared memory.
struct Shared {
    uint32_t a, b, bar0;
    uint8_t *epi;
    volatile uint32_t *tmem_slot;
    volatile int *abort_flag;
    uint32_t *again;  // two words: which of the pair's tiles to compute again
    int *first, *start;
    int stages, b_bytes;
    __device__ __forceinline__ Shared(uint8_t *raw, int stage_b_bytes)
        : stages(ring_stages(stage_b_bytes)), b_bytes(stage_b_bytes)
    {
        const uint32_t r = smem_u32(raw), base = (r + 1023u) & ~1023u;  // 128-byte swizzle atoms
        uint8_t *p = raw + (base - r);
        a = base;
        b = base + stages * kStageA;
        epi = p + kRingBytes;
        uint8_t *bars = epi + kEpiBytes;
        bar0 = smem_u32(bars);
        tmem_slot = reinterpret_cast<volatile uint32_t *>(bars + kBarBytes - 16);
        abort_flag = reinterpret_cast<volatile int *>(bars + kBarBytes - 8);
        again = reinterpret_cast<uint32_t *>(bars + kBarBytes - 32);
        first = reinterpret_cast<int *>(bars + kBarBytes);
        start = first + kMaxGroups + 2;
    }
    __device__ __forceinline__ uint32_t full(int s) const { return bar0 + 8u * s; }
    __device__ __forceinline__ uint32_t empty(int s) const { return bar0 + 8u * (kMaxStages + s); }
    __device__ __forceinline__ uint32_t ragged(int s) const { return bar0 + 8u * (2 * kMaxStages + s); }
    __device__ __forceinline__ uint32_t cleaned(int s) const { return bar0 + 8u * (3 * kMaxStages + s); }
    __device__ __forceinline__ uint32_t acc_full(int i) const { return bar0 + 8u * (4 * kMaxStages + i); }
    __device__ __forceinline__ uint32_t acc_empty(int i) const { return bar0 + 8u * (4 * kMaxStages + 2 + i); }
    __device__ __forceinline__ uint32_t drain() const { return bar0 + 8u * (4 * kMaxStages + 4); }
    __device__ __forceinline__ uint32_t stage_a(int s) const { return a + uint32_t(s * kStageA); }
    __device__ __forceinline__ uint32_t stage_b(int s) const { return b + uint32_t(s * b_bytes); }
};
static_assert(8 * (4 * kMaxStages + 5) <= kBarBytes - 32, "barrier area");

// Barriers, the groups' first positions and first units, TMEM; ends with the pair in step.
// units_of(rows): work units of a group of that many rows.  CHAIN: waits for the kernel ahead.
template <bool CHAIN, class F>
__device__ __forceinline__ uint32_t set_up(const Shared &sh, const int32_t *offsets, int groups, int64_t positions,
                                           F units_of)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < sh.stages; ++s) {
            mbar_init(sh.full(s), 1);
            mbar_init(sh.empty(s), 1);  // the MMA issuer's commit
            mbar_init(sh.ragged(s), 1);
            mbar_init(sh.cleaned(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sh.acc_full(i), 1);
            mbar_init(sh.acc_empty(i), 2 * kEpiWarps);  // the epilogue warps of both CTAs
        }
        mbar_init(sh.drain(), 1);
        *sh.abort_flag = 0;
        sh.again[0] = sh.again[1] = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    cluster_sync();  // a pair allocates TMEM together, and its barriers exist before the peer uses them
    if (warp == 1) tmem_alloc<true>(smem_u32(const_cast<uint32_t *>(sh.tmem_slot)), kTmemCols);
    if (CHAIN) chain_wait();
    else asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int g = threadIdx.x; g <= groups; g += blockDim.x)
        sh.first[g] = offsets != nullptr ? clamp_to(load_now(offsets + g), positions) : g == 0 ? 0 : int(positions);
    __syncthreads();
    if (warp == 0) {
        int carry = 0;
        for (int g0 = 0; g0 < groups; g0 += 32) {
            const int g = g0 + lane;
            int n = g < groups ? units_of(max(0, sh.first[g + 1] - sh.first[g])) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFull, n, o);
                if (lane >= o) n += v;
            }
            if (g < groups) sh.start[g + 1] = carry + n;
            carry += __shfl_sync(kFull, n, 31);
        }
        if (lane == 0) sh.start[0] = 0;
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    return *sh.tmem_slot;
}

__device__ __forceinline__ void tear_down(uint32_t tmem)
{
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves or frees TMEM while the other may still use it
    tc_fence_after();
    if ((threadIdx.x >> 5) == 1) tmem_free<true>(tmem, kTmemCols);
}

// The end of a producer: after a failure its copies get time to land before the shared memory goes
// away (they complete on the first CTA's barriers); otherwise it waits for the last release of every
// slot, so that no commit is on its way to this CTA's barriers when it exits.
__device__ __forceinline__ void finish_producer(const Shared &sh, const Watch &watch, Ring ring, bool ok)
{
    if (!ok) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 2000000ull) {
        }
        return;
    }
    for (int i = 0; i < sh.stages; ++i) {
        if (!watch.wait(sh.empty(ring.stage), ring.phase ^ 1u)) return;
        ring.next();
    }
}

// The end of an issuer that gave up: its MMAs in flight finish before TMEM is released.
__device__ __forceinline__ void drain_issuer(const Shared &sh)
{
    umma_commit<true>(sh.drain());
    const volatile int no_abort = 0;
    mbar_wait(sh.drain(), 0, &no_abort, 100000000ull);
}

// ------------------------------------------------------------------ Y = X op(W)
constexpr int kTokenWarp = 2 + kEpiWarps;
constexpr int kThreads = 32 * (kTokenWarp + 1);
constexpr int kPlain = 0, kGated = 1, kAdapted = 2;

// Rows as boxes of 128, 64, 32 and 16; gathered: rows[0] has one-row boxes.
struct TokenMaps {
    CUtensorMap rows[4];
};
// Copies `count` rows (a multiple of 16, at most 128) from row `first`, in powers of two.
__device__ __forceinline__ void load_rows(uint32_t dst, const TokenMaps &map, uint32_t bar, int column, int first, int count)
{
    int at = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (count & (128 >> i)) {
            tma_load_2d_pair(dst + 128u * at, &map.rows[i], bar, column, first + at);
            at += 128 >> i;
        }
}

struct LinearParams {
    const int32_t *offsets;
    int groups, shared_w;
    int64_t y_rows, x_rows, N;
    int ftiles, num_kb, cap;  // feature tiles of a group, K slices, tokens of a tile at most
    // splits > 1: units of a part of the K slices (and of the requests' slices) each, whose fp32 sums
    // are split_stride elements apart in Y and are added up by the next kernel
    int splits;
    int64_t split_stride;
    int y_tma;  // Y is stored to by TMA, through map_y
    const int32_t *rows;
    void *Y;
    int64_t ldy;
    int bf16;
    void *pre;
    int64_t ldp;
    // adapters: requests, and the planes of the inner products' parts (launch_shrink), each of
    // plane_rows rows of 64 ranks
    const int32_t *segments, *adapters;
    int requests, n_adapters, rank, parts;
    int plane_rows;
    const float *values;  // their fp32 values, a row of `rank` for every token
    const void *b;
    int64_t ldb, strideb;
    unsigned int *status;
    uint64_t timeout_ns;
    int inject_stall;  // test hook: the producer never fills its first slice
};

// n / d rounded up, for n up to 2^31 - 1.
__device__ __forceinline__ int parts_of(int n, int d) { return int((unsigned(n) + unsigned(d) - 1u) / unsigned(d)); }

// A unit: one feature tile of one tile of a group's tokens, over K slices [kb0, kb1).
struct LinearUnit {
    int group, feature_tile, first, tokens, width, split, kb0, kb1;
};
__device__ __forceinline__ LinearUnit linear_unit(const LinearParams &p, const Shared &sh, int u, int &group)
{
    while (u >= sh.start[group + 1]) ++group;
    const int rows = sh.first[group + 1] - sh.first[group];
    const int tiles = parts_of(rows, p.cap);
    const int width = (parts_of(rows, tiles) + 31) & ~31;  // even tiles; at most cap, none is empty
    int r = u - sh.start[group];
    LinearUnit x;
    x.split = r % p.splits;
    x.kb0 = p.num_kb * x.split / p.splits;
    x.kb1 = p.num_kb * (x.split + 1) / p.splits;
    r /= p.splits;
    const int t = r / p.ftiles;
    x.group = group;
    x.feature_tile = r - t * p.ftiles;
    x.first = sh.first[group] + t * width;
    x.tokens = min(width, rows - t * width);
    x.width = (x.tokens + 31) & ~31;
    return x;
}

// v (this lane's feature, 32 tokens) as [token][feature].
template <bool F32> __device__ __forceinline__ void stage_tokens(const float (&v)[32], uint8_t *piece, int lane, bool bf16)
{
    if (F32) {
        float *t = reinterpret_cast<float *>(piece);
#pragma unroll
        for (int i = 0; i < 32; ++i) t[i * 32 + lane] = v[i];
    } else {
        uint16_t *t = reinterpret_cast<uint16_t *>(piece);
#pragma unroll
        for (int i = 0; i < 32; ++i) t[i * 32 + lane] = to_16(v[i], bf16);
    }
}

// 32 tokens of this warp's 32 features to rows `first` .. of an array in 16-byte pieces of token rows,
// the first `tokens` of them: for the last tokens of a group, whose 32 rows are not all its own, and for
// arrays that TMA cannot store to.
template <bool F32>
__device__ __forceinline__ void store_tokens(const float (&v)[32], uint8_t *tile, int lane, uint8_t *base, int64_t ld_bytes,
                                             int first, int tokens, int64_t feature0, int64_t N, bool bf16)
{
    constexpr int kSize = F32 ? 4 : 2, kPieces = 2 * kSize;  // 16-byte pieces of 32 features
    constexpr int kPasses = kPieces;                         // 32 / kPieces tokens a pass
    __syncwarp();
    stage_tokens<F32>(v, tile, lane, bf16);
    __syncwarp();
    const int piece = lane % kPieces, i0 = lane / kPieces;
    uint4 q[kPasses];
#pragma unroll
    for (int j = 0; j < kPasses; ++j)
        q[j] = *reinterpret_cast<const uint4 *>(tile + (j * 32 + lane) * 16);
    const int64_t f = feature0 + piece * (16 / kSize);
    uint8_t *dst = base + int64_t(first + i0) * ld_bytes + f * kSize;
    if (f + 16 / kSize <= N) {
#pragma unroll
        for (int j = 0; j < kPasses; ++j, dst += (32 / kPieces) * ld_bytes)
            if (i0 + j * (32 / kPieces) < tokens) *reinterpret_cast<uint4 *>(dst) = q[j];
    } else if (f < N) {
#pragma unroll 1
        for (int j = 0; j < kPasses; ++j, dst += (32 / kPieces) * ld_bytes) {
            if (i0 + j * (32 / kPieces) >= tokens) break;
            const uint16_t *e = reinterpret_cast<const uint16_t *>(tile + (j * 32 + lane) * 16);
            for (int c = 0; c < int(N - f) * kSize / 2; ++c) reinterpret_cast<uint16_t *>(dst)[c] = e[c];
        }
    }
}

__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }

// Whether the tensor cores cannot form a request's product: an adapter's rows of B for a tile of 256
// features hold an infinity or NaN, or a finite inner product of tokens [t0, t1) has an infinite part.
__device__ __noinline__ bool unfit(const LinearParams &p, int adapter, int feature_tile, int t0, int t1, int lane)
{
    const uint32_t exponent = p.bf16 ? 0x7f80u : 0x7c00u;  // all ones: no finite number
    const int64_t f0 = int64_t(feature_tile) * 256;
    const int rows = int(min(p.N - f0, int64_t(256))), pieces = (p.rank + 7) / 8;
    const uint16_t *b = static_cast<const uint16_t *>(p.b) + adapter * p.strideb + f0 * p.ldb;
    bool found = false;
    for (int i = lane; i < rows * pieces; i += 32) {
        const uint4 v = load_tail(b + i / pieces * p.ldb, i % pieces * 8, p.rank);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) found |= (w[c] & exponent) == exponent || ((w[c] >> 16) & exponent) == exponent;
    }
    for (int64_t i = int64_t(t0) * p.rank + lane; i < int64_t(t1) * p.rank; i += 32) {
        const float v = __ldcg(p.values + i);
        found |= fabsf(v) <= FLT_MAX && (to_16(v, p.bf16) & exponent) == exponent;
    }
    return __any_sync(kFull, found);
}

// The requests that share a tile's tokens and have an adapter, in order, those of the unit's split of
// them; the roles' warps walk them in step, 32 requests looked up at a time.
//
// A request's slices: for every 64 ranks, its inner products' parts in turn, as many parts behind one
// another in the token half of a stage as fit (all of them for a short request), each multiplied with
// the same adapter rows.
//
// The columns of a request's slices are whole blocks of 32, in which other requests' tokens are zeros, so
// an infinity or NaN among the adapter's rows would make NaN of them; and fp16's parts of an inner product
// beyond 65504, or bf16's of one close to fp32's largest, are infinite though their value is not.  A tile whose sums are not all
// finite is computed a second time (`careful`), in which requests whose product is unfit for the tensor
// cores are left out of the slices and added to the sums by the epilogue (add_late).  What the other
// requests get does not depend on them in a bit: the same slices in the same order.  Where all values are
// finite this costs about 1 us a call; 8192 tokens, rank 64, 4096 x 4096 take 204 us, 923 with an infinity
// in one of 7 requests' adapters and 4.8 ms with one in all of them.
struct TileRequests {
    const LinearParams &p;
    int t0, t1, q0, lane, skip, feature_tile;
    bool careful;
    unsigned left, late;  // of the 32 requests at q0: those to come, those left out of the slices
    int lo, hi, ad;  // of request q0 + lane: its tokens within the tile and its adapter
    __device__ __forceinline__ TileRequests(const LinearParams &params, const LinearUnit &x, int l, bool second)
        : p(params), t0(x.first), t1(x.first + x.tokens), lane(l), skip(x.split), feature_tile(x.feature_tile), careful(second)
    {
        // requests that end at or before the tile's first token, 32 candidates at a time: whole runs,
        // then the run that is left
        q0 = 0;
        for (int n = p.requests; n > 0;) {
            const int run = (n + 31) / 32, last = (lane + 1) * run - 1;
            const bool done = last < n && clamp_to(load_now(p.segments + q0 + last + 1), p.y_rows) <= t0;
            const int c = __popc(__ballot_sync(kFull, done));
            q0 += c * run;
            n = (c + 1) * run <= n ? run - 1 : n - c * run;
        }
        look_up();
    }
    __device__ __forceinline__ void look_up()
    {
        const int q = q0 + lane;
        lo = hi = 0;
        ad = -1;
        if (q < p.requests) {
            lo = max(clamp_to(load_now(p.segments + q), p.y_rows), t0);
            hi = min(clamp_to(load_now(p.segments + q + 1), p.y_rows), t1);
            ad = load_now(p.adapters + q);
        }
        left = __ballot_sync(kFull, lo < hi && unsigned(ad) < unsigned(p.n_adapters));
        late = 0u;
        if (careful)
            for (unsigned look = left; look != 0u; look &= look - 1u) {
                const int at = __ffs(look) - 1;
                if (unfit(p, __shfl_sync(kFull, ad, at), feature_tile, __shfl_sync(kFull, lo, at), __shfl_sync(kFull, hi, at), lane))
                    late |= 1u << at;
            }
        more = __any_sync(kFull, q == q0 + 31 && q + 1 < p.requests && clamp_to(load_now(p.segments + q + 1), p.y_rows) < t1);
    }
    bool more;
    // Next of the split's requests, by its lane.
    __device__ __forceinline__ bool advance(int &at)
    {
        for (;; --skip) {
            while (left == 0u) {
                if (!more) return false;
                q0 += 32;
                look_up();
            }
            if (skip == 0) break;
            left &= left - 1u;
        }
        skip = p.splits - 1;
        at = __ffs(left) - 1;
        left &= left - 1u;
        return true;
    }
    // Next request that is left out: its adapter and its tokens within the tile.
    __device__ __forceinline__ bool next_late(int &adapter, int &first, int &end)
    {
        int at;
        do {
            if (!advance(at)) return false;
        } while (!((late >> at) & 1u));
        adapter = __shfl_sync(kFull, ad, at);
        first = __shfl_sync(kFull, lo, at);
        end = __shfl_sync(kFull, hi, at);
        return true;
    }
    // Next request with slices: its adapter, the columns [c0, c0 + n) of the tile that hold its tokens,
    // multiples of 32, and the first of the rows of its inner products.
    __device__ __forceinline__ bool next(int &adapter, int &c0, int &n, int &row)
    {
        int at;
        do {
            if (!advance(at)) return false;
        } while ((late >> at) & 1u);
        adapter = __shfl_sync(kFull, ad, at);
        const int b0 = __shfl_sync(kFull, lo, at) / 32, b1 = (__shfl_sync(kFull, hi, at) + 31) / 32;
        c0 = b0 * 32 - t0;
        n = (b1 - b0) * 32;
        row = (b0 + q0 + at) * 32;
        return true;
    }
    // Parts in one slice of a request of n columns.
    __device__ __forceinline__ int parts_a_slice(int n) const { return max(1, min(p.parts, p.cap / n)); }
};

// Looked up at a unit's start, while its first slices are on their way; the other forms have none.
struct NoRequests {
    __device__ __forceinline__ NoRequests(const LinearParams &, const LinearUnit &, int, bool) {}
    __device__ __forceinline__ bool next(int &, int &, int &, int &) { return false; }
    __device__ __forceinline__ int parts_a_slice(int) const { return 1; }
};
template <int EPI> using RequestsOf = typename std::conditional<EPI == kAdapted, TileRequests, NoRequests>::type;

// Adds the products of the requests that a tile's second computation leaves out to `sums`, 32 tokens from
// `first` of the lane's feature f + lane as [token][lane]: fp32 values and sums, as the few-rows kernel's.
__device__ __noinline__ void add_late(const LinearParams &p, const LinearUnit x, float *sums, int first, int tokens, int64_t f,
                                      int lane)
{
    TileRequests requests(p, x, lane, true);
    int adapter, t0, t1;
    while (requests.next_late(adapter, t0, t1)) {
        if (f + lane >= p.N) continue;
        const uint16_t *b = static_cast<const uint16_t *>(p.b) + adapter * p.strideb + (f + lane) * p.ldb;
        for (int t = max(t0, first); t < min(t1, first + min(tokens, 32)); ++t) {
            const float *values = p.values + int64_t(t) * p.rank;
            float low = 0.0f;
            for (int j = 0; j < p.rank; j += 8) {
                const uint4 e = load_tail(b, j, p.rank);
                const uint32_t w[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint16_t u = uint16_t(w[c / 2] >> (16 * (c & 1)));
                    const float v = p.bf16 ? __bfloat162float(__ushort_as_bfloat16(u)) : __half2float(__ushort_as_half(u));
                    if (j + c < p.rank) low = fmaf(v, __ldcg(values + j + c), low);
                }
            }
            sums[(t - first) * 32 + lane] += low;
        }
    }
}

// The tiles that the pair computes again, by their number modulo 64: those that the epilogue of either CTA
// noted; none after a failure.  Both CTAs come here with all threads and get the same.
__device__ __forceinline__ uint64_t tiles_again(const Shared &sh)
{
    __syncwarp();
    cluster_sync();
    uint64_t all = 0;
    uint32_t stop = 0;
#pragma unroll
    for (uint32_t r = 0; r < 2; ++r) {
        uint32_t lo, hi, flag;
        const uint32_t at = map_to_rank(smem_u32(sh.again), r);
        const uint32_t abort_at = map_to_rank(smem_u32(const_cast<int *>(sh.abort_flag)), r);
        asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(lo), "=r"(hi) : "r"(at) : "memory");
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(flag) : "r"(abort_at) : "memory");
        all |= uint64_t(hi) << 32 | lo;
        stop |= flag;
    }
    return stop != 0u ? 0ull : all;
}

// W_MN: W stored K x N (features contiguous).
//
// Bound by the tensor pipe (75% active) and the power limit where groups are large: 32 groups of 512 rows,
// N = K = 2048, bf16, 87.6 us (1569 TFLOP/s, 0.81 of the measured burst peak), the last wave of tiles
// being 4% of it.  Gated, 1024 outputs of 2048 weight rows, 89.9 us (1529 TFLOP/s, 72% active).  8192 tokens
// with adapters of rank 64, 4096 x 4096: 157 us (1750 TFLOP/s of the projection alone).
//
// Every output is rounded once, from fp32.  Y in 16 bits between an expert's two products is a choice for
// the second one's tensor cores, which read 16-bit rows: the error of the layer's output is 1.41 times that
// of its own rounding.  An fp32 Y is to be had where no product reads it.
template <int W_MN, int EPI, bool Y_F32>
__global__ void __launch_bounds__(kThreads, 1)
grouped_linear_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ TokenMaps map_x,
                      const __grid_constant__ CUtensorMap map_b, const __grid_constant__ TokenMaps map_inner,
                      const __grid_constant__ CUtensorMap map_y, const __grid_constant__ LinearParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const Shared sh(smem_raw, p.cap * 64);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int cap = p.cap, ftiles = p.ftiles * p.splits;
    const uint32_t tmem = set_up<EPI != kAdapted>(sh, p.offsets, p.groups, p.y_rows,
                                 [=](int rows) { return parts_of(rows, cap) * ftiles; });
    const Watch watch{sh.abort_flag, p.status, p.timeout_ns};
    const int units = sh.start[p.groups], unit0 = int(cluster_id_x()), step = int(cluster_count_x());
    constexpr int kFeatures = EPI == kGated ? 128 : 256;  // of a unit
    const int blocks = EPI == kAdapted ? (p.rank + 63) / 64 : 1;  // of 64 ranks

    // A role's place in the ring and the accumulators; with adapters it may go through its tiles twice.
    Ring ring(sh.stages);
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    uint64_t again = ~0ull;
    auto wanted = [&](int n) { return EPI != kAdapted || ((again >> (n & 63)) & 1u) != 0u; };
    for (bool careful = false;; careful = true) {
        if (warp == 0) {
            // ---------------- weight producer (warps in step, one elected lane copying)
            const bool leader = elect_one();
            const uint32_t full0 = map_to_rank(sh.full(0), 0);  // the first CTA's
            int group = 0;
            if (leader) tma_prefetch_desc(&map_w);
            for (int u = unit0, n = 0; ok && u < units; u += step, ++n) {
                if (!wanted(n)) continue;
                const LinearUnit x = linear_unit(p, sh, u, group);
                RequestsOf<EPI> requests(p, x, lane, careful);
                const int f0 = x.feature_tile * kFeatures + int(rank) * (kFeatures / 2);
                const int wg = p.shared_w ? 0 : x.group;
                const uint32_t bytes = 2u * (kStageA + uint32_t(x.width) * 64u);
                for (int kb = x.kb0; kb < x.kb1; ++kb) {
                    ok = watch.wait(sh.empty(ring.stage), ring.phase ^ 1u);
                    if (__any_sync(kFull, !ok)) {
                        ok = false;
                        break;
                    }
                    if (leader) {
                        if (rank == 0) mbar_expect_tx(sh.full(ring.stage), bytes);
                        if (!(p.inject_stall && kb == x.kb0 && u == unit0)) {
                            const uint32_t full = full0 + 8u * ring.stage, a = sh.stage_a(ring.stage);
                            if (W_MN) {  // two boxes of 64 features x 64 k
                                tma_load_3d_pair(a, &map_w, full, f0, kb * 64, wg);
                                tma_load_3d_pair(a + 8192, &map_w, full, f0 + 64, kb * 64, wg);
                            } else if (EPI == kGated) {  // 64 gate rows and their up rows
                                tma_load_3d_pair(a, &map_w, full, kb * 64, f0, wg);
                                tma_load_3d_pair(a + 8192, &map_w, full, kb * 64, int(p.N) + f0, wg);
                            } else {
                                tma_load_3d_pair(a, &map_w, full, kb * 64, f0, wg);
                            }
                        }
                    }
                    __syncwarp();
                    ring.next();
                }
                if (EPI == kAdapted && ok) {
                    int ad, c0, cols, row;
                    while (ok && requests.next(ad, c0, cols, row)) {
                        const int most = requests.parts_a_slice(cols);
                        for (int r0 = 0, i = 0; ok && r0 < p.rank; (i += most) >= p.parts ? (i = 0, r0 += 64) : 0) {
                            ok = watch.wait(sh.empty(ring.stage), ring.phase ^ 1u);
                            if (__any_sync(kFull, !ok)) {
                                ok = false;
                                break;
                            }
                            if (leader) {
                                const uint32_t rows = uint32_t(cols) * uint32_t(min(most, p.parts - i));
                                if (rank == 0) mbar_expect_tx(sh.full(ring.stage), 2u * (kStageA + rows * 64u));
                                tma_load_3d_pair(sh.stage_a(ring.stage), &map_b, full0 + 8u * ring.stage, r0, f0, ad);
                            }
                            __syncwarp();
                            ring.next();
                        }
                    }
                }
            }
            if (leader) finish_producer(sh, watch, ring, ok);
        } else if (warp == kTokenWarp) {
            // ---------------- token producer
            const bool leader = elect_one();
            const uint32_t full0 = map_to_rank(sh.full(0), 0);
            int group = 0;
            if (leader) tma_prefetch_desc(&map_x.rows[0]);
            for (int u = unit0, n = 0; ok && u < units; u += step, ++n) {
                if (!wanted(n)) continue;
                const LinearUnit x = linear_unit(p, sh, u, group);
                RequestsOf<EPI> requests(p, x, lane, careful);
                const int half = x.width / 2;                     // tokens this CTA loads
                const unsigned row0 = unsigned(x.first) + rank * half, end = x.first + x.tokens;  // row0: past 2^31 too
                int4 from = make_int4(0, 0, 0, 0);
                if (p.rows != nullptr && 4 * lane < half) {       // a row outside x is read as zeros
                    int r[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const unsigned q = row0 + 4 * lane + i;
                        r[i] = q < end ? load_now(p.rows + q) : -1;
                        if (r[i] < 0 || r[i] >= p.x_rows) r[i] = int(p.x_rows);
                    }
                    from = make_int4(r[0], r[1], r[2], r[3]);
                }
                for (int kb = x.kb0; kb < x.kb1; ++kb) {
                    ok = watch.wait(sh.empty(ring.stage), ring.phase ^ 1u);
                    if (__any_sync(kFull, !ok)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = full0 + 8u * ring.stage, b = sh.stage_b(ring.stage);
                    if (p.rows != nullptr) {
                        if (4 * lane < half) tma_gather4_pair(b + 512u * lane, &map_x.rows[0], full, kb * 64, from);
                    } else if (leader) {
                        load_rows(b, map_x, full, kb * 64, int(row0), half);
                    }
                    __syncwarp();
                    ring.next();
                }
                if (EPI == kAdapted && ok) {
                    // the inner products come from the kernel ahead, which itself waited for what x comes from
                    asm volatile("griddepcontrol.wait;" ::: "memory");
                    int ad, c0, cols, row;
                    while (ok && requests.next(ad, c0, cols, row)) {
                        const int most = requests.parts_a_slice(cols);
                        for (int r0 = 0, i = 0; ok && r0 < p.rank; (i += most) >= p.parts ? (i = 0, r0 += 64) : 0) {
                            ok = watch.wait(sh.empty(ring.stage), ring.phase ^ 1u);
                            if (__any_sync(kFull, !ok)) {
                                ok = false;
                                break;
                            }
                            if (leader)
                                for (int j = 0; j < most && i + j < p.parts; ++j)
                                    load_rows(sh.stage_b(ring.stage) + uint32_t(j * cols) * 64u, map_inner, full0 + 8u * ring.stage, 0,
                                              ((i + j) * blocks + r0 / 64) * p.plane_rows + row + int(rank) * (cols / 2), cols / 2);
                            __syncwarp();
                            ring.next();
                        }
                    }
                }
            }
            if (leader && !ok) finish_producer(sh, watch, ring, false);
            // a CTA without tiles of its own still orders this launch behind the one ahead of it
            if (EPI == kAdapted) asm volatile("griddepcontrol.wait;" ::: "memory");
        } else if (warp == 1) {
            if (rank == 0) {
                // ---------------- MMA issuer: the warp in step, one elected lane issuing
                const bool leader = elect_one();
                const uint32_t fmt = p.bf16 ? (1u << 7) | (1u << 10) : 0u;
                // descriptors of stage 0; a later stage or K step only moves the start address
                const uint64_t a0 = W_MN ? smem_desc(sh.a, 8192, 1024) : smem_desc(sh.a, 16, 1024);
                const uint64_t b0 = smem_desc(sh.b, 16, 1024);
                constexpr uint64_t kStepA = W_MN ? 2048 >> 4 : 32 >> 4, kStepB = 32 >> 4;
                int group = 0;
                for (int u = unit0, n = 0; ok && u < units; u += step, ++n) {
                    if (!wanted(n)) continue;
                    const LinearUnit x = linear_unit(p, sh, u, group);
                    RequestsOf<EPI> requests(p, x, lane, careful);
                    const uint32_t idesc = make_idesc(W_MN, 0, x.width, 256) | fmt;
                    ok = watch.wait<true>(sh.acc_empty(acc), acc_phase ^ 1u);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + uint32_t(acc * kAccCols);
                    for (int kb = x.kb0; kb < x.kb1; ++kb) {
                        ok = watch.wait(sh.full(ring.stage), ring.phase);
                        if (!ok) break;
                        tc_fence_after();
                        if (leader) {
                            const uint64_t a = a0 + uint32_t(ring.stage * (kStageA >> 4));
                            const uint64_t b = b0 + uint32_t(ring.stage * (sh.b_bytes >> 4));
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                umma_f16<true>(d, a + k * kStepA, b + k * kStepB, idesc, kb > x.kb0 || k > 0 ? 1u : 0u);
                            commit_both(sh.empty(ring.stage));
                        }
                        __syncwarp();
                        ring.next();
                    }
                    if (EPI == kAdapted && ok) {
                        int ad, c0, cols, row;
                        while (ok && requests.next(ad, c0, cols, row)) {
                            const uint32_t part_idesc = make_idesc(0, 0, cols, 256) | fmt;
                            const int most = requests.parts_a_slice(cols);
                            for (int r0 = 0, i = 0; r0 < p.rank; (i += most) >= p.parts ? (i = 0, r0 += 64) : 0) {
                                ok = watch.wait(sh.full(ring.stage), ring.phase);
                                if (!ok) break;
                                tc_fence_after();
                                if (leader) {
                                    const uint64_t a = a0 + uint32_t(ring.stage * (kStageA >> 4));
                                    uint64_t b = b0 + uint32_t(ring.stage * (sh.b_bytes >> 4));
                                    const int steps = (p.rank - r0 + 15) / 16;
                                    for (int j = 0; j < most && i + j < p.parts; ++j, b += uint32_t(cols * 64) >> 4) {
#pragma unroll
                                        for (int k = 0; k < 4; ++k)
                                            if (k < steps)
                                                umma_f16<true>(d + uint32_t(c0), a + k * kStepA, b + k * kStepB, part_idesc, 1u);
                                    }
                                    commit_both(sh.empty(ring.stage));
                                }
                                __syncwarp();
                                ring.next();
                            }
                        }
                    }
                    if (!ok) break;
                    if (leader) commit_both(sh.acc_full(acc));
                    if (++acc == 2) {
                        acc = 0;
                        acc_phase ^= 1u;
                    }
                }
                if (!ok && leader) drain_issuer(sh);
            }
        } else {
            // ---------------- epilogue: TMEM lanes 32 * quarter .. of this CTA's 128 rows
            const int quarter = warp & 3, half = (warp - 2) >> 2;
            uint8_t *tile = sh.epi + (warp - 2) * 4096;
            Staging<Y_F32> staging(tile, lane);
            int group = 0;
            const uint32_t acc_empty0 = map_to_rank(sh.acc_empty(0), 0);
            const int64_t ldy = p.ldy * (Y_F32 ? 4 : 2);
            auto put = [&](const float (&v)[32], int first, int tokens, int64_t f, int split) {
                if (f >= p.N) return;
                if (p.y_tma && tokens >= 32) {
                    uint8_t *piece = staging.next();
                    stage_tokens<Y_F32>(v, piece, lane, p.bf16);
                    staging.store(&map_y, piece, int(f), first, split);
                } else {
                    uint8_t *Y = static_cast<uint8_t *>(p.Y) + split * p.split_stride * (Y_F32 ? 4 : 2);
                    store_tokens<Y_F32>(v, staging.all(), lane, Y, ldy, first, tokens, f, p.N, p.bf16);
                }
            };
            for (int u = unit0, n = 0; u < units; u += step, ++n) {
                if (!wanted(n)) continue;
                const LinearUnit x = linear_unit(p, sh, u, group);
                const bool got = mbar_wait(sh.acc_full(acc), acc_phase, sh.abort_flag, p.timeout_ns);
                if (epilogue_any<kEpiWarps>(!got)) {  // the warps give up together
                    watch.raise();
                    break;
                }
                tc_fence_after();
                const uint32_t taddr = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(acc * kAccCols);
                if (EPI == kGated) {
                    // quarters 0, 1 hold gate rows, 2, 3 the up rows of the same features; of two
                    // pieces of 32 tokens the gate's warp finishes the first, the up's warp the second
                    const bool up = quarter >= 2;
                    const int64_t f = int64_t(x.feature_tile) * 128 + int64_t(rank) * 64 + (quarter & 1) * 32;
                    const int meet = 2 + 2 * half + (quarter & 1);  // named barrier of the two warps
                    float *own = reinterpret_cast<float *>(tile);
                    const float *other = reinterpret_cast<const float *>(sh.epi + ((warp - 2) ^ 2) * 4096);
                    if (64 * half >= x.width) release_accumulator(acc_empty0 + 8u * acc, lane);
#pragma unroll 1
                    for (int c = 64 * half; c < x.width; c += 128) {
                        const bool two = c + 32 < x.width;
                        float v0[32], v1[32];
                        __syncwarp();
                        tmem_ld_32(taddr + c, v0);
                        if (two) tmem_ld_32(taddr + c + 32, v1);
                        if (c + 128 >= x.width) release_accumulator(acc_empty0 + 8u * acc, lane);
                        staging.all();
                        if (p.pre != nullptr) {
                            uint8_t *pre = static_cast<uint8_t *>(p.pre) + (up ? p.N * 2 : 0);
                            if (f + 32 <= p.N && p.N % 8 == 0) {
                                store_tokens<false>(v0, tile, lane, pre, p.ldp * 2, x.first + c, x.tokens - c, f, p.N, p.bf16);
                                if (two)
                                    store_tokens<false>(v1, tile, lane, pre, p.ldp * 2, x.first + c + 32, x.tokens - c - 32, f,
                                                        p.N, p.bf16);
                            } else if (f + lane < p.N) {  // the up half's pieces may not be 16-byte aligned
                                uint16_t *dst = reinterpret_cast<uint16_t *>(pre) + int64_t(x.first + c) * p.ldp + f + lane;
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    if (c + i < x.tokens) dst[i * p.ldp] = to_16(v0[i], p.bf16);
                                    if (two && c + 32 + i < x.tokens) dst[(32 + i) * p.ldp] = to_16(v1[i], p.bf16);
                                }
                            }
                        }
                        __syncwarp();
                        if (up) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) own[i * 32 + lane] = v0[i];
                        } else if (two) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) own[i * 32 + lane] = v1[i];
                        }
                        asm volatile("bar.sync %0, 64;" ::"r"(meet) : "memory");
                        if (!up) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v0[i] = silu(v0[i]) * other[i * 32 + lane];
                        } else if (two) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v0[i] = silu(other[i * 32 + lane]) * v1[i];
                        }
                        asm volatile("bar.sync %0, 64;" ::"r"(meet) : "memory");
                        const int at = up ? c + 32 : c;
                        if (!up || two) put(v0, x.first + at, x.tokens - at, f, 0);
                    }
                } else {
                    const int64_t f = int64_t(x.feature_tile) * 256 + int64_t(rank) * 128 + quarter * 32;
                    if (32 * half >= x.width) release_accumulator(acc_empty0 + 8u * acc, lane);
#pragma unroll 1
                    for (int c = 32 * half; c < x.width; c += 64) {
                        float v[32];
                        __syncwarp();
                        tmem_ld_32(taddr + c, v);
                        if (c + 64 >= x.width) release_accumulator(acc_empty0 + 8u * acc, lane);
                        if (EPI == kAdapted && !careful) {
                            bool finite = true;
#pragma unroll
                            for (int i = 0; i < 32; ++i) finite = finite && fabsf(v[i]) <= FLT_MAX;
                            if (__any_sync(kFull, !finite) && lane == 0) atomicOr(sh.again + ((n >> 5) & 1), 1u << (n & 31));
                        } else if (EPI == kAdapted) {
                            float *sums = reinterpret_cast<float *>(staging.all());
#pragma unroll
                            for (int i = 0; i < 32; ++i) sums[i * 32 + lane] = v[i];
                            __syncwarp();
                            add_late(p, x, sums, x.first + c, x.tokens - c, f, lane);
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = sums[i * 32 + lane];
                            __syncwarp();
                        }
                        put(v, x.first + c, x.tokens - c, f, x.split);
                    }
                }
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            staging.finish();
        }
        if (EPI != kAdapted || careful || (again = tiles_again(sh)) == 0u) break;
        asm volatile("griddepcontrol.wait;" ::: "memory");
    }
    tear_down(tmem);
}

// ------------------------------------------------------------------ dW = dY^T X
constexpr int kCleaner = kTokenWarp + 1;  // warp
constexpr int kGradThreads = kThreads + 32;

struct GradParams {
    const int32_t *offsets;
    int groups;
    int64_t positions, N, K;
    int ntiles, ktiles;
    void *dW;
    int64_t lddw, stridedw;
    int dw_tma;  // dW is stored to by TMA, through map_dw
    int bf16;
    unsigned int *status;
    uint64_t timeout_ns;
    int inject_stall;
};

struct GradUnit {
    int group, tn, tk, first, rows;
};
__device__ __forceinline__ GradUnit grad_unit(const GradParams &p, const Shared &sh, int u)
{
    // every group has the same number of units
    const int per = p.ntiles * p.ktiles, g = u / per, r = u - g * per;
    return GradUnit{g, r / p.ktiles, r % p.ktiles, sh.first[g], max(0, sh.first[g + 1] - sh.first[g])};
}

// First position, within the group, of a unit's i-th slice: the ragged one, if there is one, comes first,
// so that part of its way through the cleaners passes while the slices of the unit before it are
// multiplied (32 groups of 1023 rows, 2048 x 1024: 94 us, 3% more with it last; of 1024 rows 82 us).
__device__ __forceinline__ int slice_start(int rows, int i)
{
    return (rows & 63) == 0 ? i * 64 : i == 0 ? rows & ~63 : (i - 1) * 64;
}

// A pair's tile is 256 (n) x 256 (k): each CTA holds 128 columns of dY and 128 of X as two boxes of
// 64 columns x 64 positions each.  A whole slice lands on the first CTA's full barrier; a group's last
// one on each CTA's own ragged barrier, from which the cleaners pass it on: the second CTA's to the
// first's (cleaned), the first's to the full barrier.
//
// Bound by the tensor pipe (71% active) and the stores of dW: 32 groups of 512 positions, 2048 x 2048, 16-bit
// dW, 89.7 us (1533 TFLOP/s, each input read once).
template <bool DW_F32>
__global__ void __launch_bounds__(kGradThreads, 1)
grouped_grad_kernel(const __grid_constant__ CUtensorMap map_dy, const __grid_constant__ CUtensorMap map_x,
                    const __grid_constant__ CUtensorMap map_dw, const GradParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const Shared sh(smem_raw, kMaxStageB);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const uint32_t tmem = set_up<true>(sh, p.offsets, p.groups, p.positions, [](int) { return 0; });
    const Watch watch{sh.abort_flag, p.status, p.timeout_ns};
    const int units = p.groups * p.ntiles * p.ktiles, unit0 = int(cluster_id_x()), step = int(cluster_count_x());
    constexpr uint32_t kSliceBytes = kStageA + kMaxStageB;

    if (warp == 0 || warp == kTokenWarp) {
        // ---------------- producers, of dY and of X (warps in step, one elected lane copying)
        const bool leader = elect_one(), of_x = warp != 0;
        const CUtensorMap *map = of_x ? &map_x : &map_dy;
        const uint32_t full0 = map_to_rank(sh.full(0), 0), ragged0 = map_to_rank(sh.ragged(0), rank);
        Ring ring(sh.stages);
        bool ok = true;
        if (leader) tma_prefetch_desc(map);
        for (int u = unit0; ok && u < units; u += step) {
            const GradUnit x = grad_unit(p, sh, u);
            const int c0 = (of_x ? x.tk : x.tn) * 256 + int(rank) * 128;
            for (int i = 0; i < parts_of(x.rows, 64); ++i) {
                const int s = slice_start(x.rows, i);
                ok = watch.wait(sh.empty(ring.stage), ring.phase ^ 1u);
                if (__any_sync(kFull, !ok)) {
                    ok = false;
                    break;
                }
                if (leader) {
                    const bool ragged = x.rows - s < 64;  // lands on this CTA's own barrier, for its cleaner
                    const uint32_t bar = (ragged ? ragged0 : full0) + 8u * ring.stage;
                    if (!of_x) {
                        if (ragged) mbar_expect_tx(sh.ragged(ring.stage), kSliceBytes);
                        else if (rank == 0) mbar_expect_tx(sh.full(ring.stage), 2 * kSliceBytes);
                    }
                    if (!(p.inject_stall && i == 0 && u == unit0)) {
                        const uint32_t dst = of_x ? sh.stage_b(ring.stage) : sh.stage_a(ring.stage);
                        tma_load_2d_pair(dst, map, bar, c0, x.first + s);
                        tma_load_2d_pair(dst + 8192, map, bar, c0 + 64, x.first + s);
                    }
                }
                __syncwarp();
                ring.next();
            }
        }
        if (leader && (!ok || !of_x)) finish_producer(sh, watch, ring, ok);
    } else if (warp == 1) {
        if (rank == 0) {
            // ---------------- MMA issuer
            const bool leader = elect_one();
            const uint32_t idesc = make_idesc(1, 1, 256, 256) | (p.bf16 ? (1u << 7) | (1u << 10) : 0u);
            const uint64_t a0 = smem_desc(sh.a, 8192, 1024), b0 = smem_desc(sh.b, 8192, 1024);
            Ring ring(sh.stages);
            int acc = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            for (int u = unit0; ok && u < units; u += step) {
                const GradUnit x = grad_unit(p, sh, u);
                if (x.rows == 0) continue;  // the epilogue writes zeros by itself
                ok = watch.wait<true>(sh.acc_empty(acc), acc_phase ^ 1u);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + uint32_t(acc * kAccCols);
                for (int i = 0; i < parts_of(x.rows, 64); ++i) {
                    const int s = slice_start(x.rows, i);
                    ok = watch.wait(sh.full(ring.stage), ring.phase);
                    if (!ok) break;
                    tc_fence_after();
                    if (leader) {
                        const uint64_t a = a0 + uint32_t(ring.stage * (kStageA >> 4));
                        const uint64_t b = b0 + uint32_t(ring.stage * (kMaxStageB >> 4));
                        const int steps = min(4, parts_of(x.rows - s, 16));  // 16 positions an MMA
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < steps)
                                umma_f16<true>(d, a + k * (2048 >> 4), b + k * (2048 >> 4), idesc, i > 0 || k > 0 ? 1u : 0u);
                        commit_both(sh.empty(ring.stage));
                    }
                    __syncwarp();
                    ring.next();
                }
                if (!ok) break;
                if (leader) commit_both(sh.acc_full(acc));
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            if (!ok && leader) drain_issuer(sh);
        }
    } else if (warp == kCleaner) {
        // ---------------- cleaner: zeros for the positions behind the group's last, up to the MMA's
        // granularity of 16
        Ring ring(sh.stages);
        uint32_t parity = 0;  // of each stage's ragged and cleaned barriers, one bit a stage
        bool ok = true;
        for (int u = unit0; ok && u < units; u += step) {
            const GradUnit x = grad_unit(p, sh, u);
            for (int i = 0; i < parts_of(x.rows, 64); ++i) {
                const int left = x.rows - slice_start(x.rows, i);
                if (left < 64) {
                    bool got = true;
                    if (lane == 0) got = watch.wait(sh.ragged(ring.stage), (parity >> ring.stage) & 1u);
                    if (__any_sync(kFull, !got)) {
                        ok = false;
                        break;
                    }
                    const int end = (left + 15) & ~15, pieces = (end - left) * 8;  // 16-byte pieces of a box
                    const uint32_t a = sh.stage_a(ring.stage), b = sh.stage_b(ring.stage);
                    for (int q = lane; q < 4 * pieces; q += 32) {
                        const int box = q / pieces;
                        const uint32_t at = (box < 2 ? a : b) + (box & 1) * 8192u + uint32_t(left) * 128u +
                                            uint32_t(q - box * pieces) * 16u;
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0u) : "memory");
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    got = true;
                    if (lane == 0) {
                        if (rank == 1) {
                            mbar_arrive_cluster(map_to_rank(sh.cleaned(ring.stage), 0));
                        } else {
                            got = watch.wait<true>(sh.cleaned(ring.stage), (parity >> ring.stage) & 1u);
                            if (got) mbar_arrive(sh.full(ring.stage));
                        }
                    }
                    if (__any_sync(kFull, !got)) {
                        ok = false;
                        break;
                    }
                    parity ^= 1u << ring.stage;
                }
                ring.next();
            }
        }
    } else {
        // ---------------- epilogue: TMEM lane = row of dW; 32 x 32 pieces pass through the staging tile
        // to TMA stores or, where TMA cannot store, to 128- or 64-byte row segments
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        float4 *tile = reinterpret_cast<float4 *>(sh.epi + (warp - 2) * 4096);
        Staging<DW_F32> staging(sh.epi + (warp - 2) * 4096, lane);
        const uint32_t acc_empty0 = map_to_rank(sh.acc_empty(0), 0);
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int u = unit0; u < units; u += step) {
            const GradUnit x = grad_unit(p, sh, u);
            if (x.rows > 0) {
                const bool got = mbar_wait(sh.acc_full(acc), acc_phase, sh.abort_flag, p.timeout_ns);
                if (epilogue_any<kEpiWarps>(!got)) {
                    watch.raise();
                    break;
                }
                tc_fence_after();
            }
            const uint32_t taddr = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(acc * kAccCols);
            const int64_t n0 = int64_t(x.tn) * 256 + int64_t(rank) * 128 + quarter * 32;
#pragma unroll 1
            for (int c = 32 * half; c < 256; c += 64) {
                const int64_t k0 = int64_t(x.tk) * 256 + c;
                float v[32];
                __syncwarp();
                if (x.rows > 0) {
                    tmem_ld_32(taddr + c, v);
                    if (c + 64 >= 256) release_accumulator(acc_empty0 + 8u * acc, lane);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0.0f;
                }
                if (k0 >= p.K || n0 >= p.N) continue;
                if (p.dw_tma) {  // laid out as the tensor map's 128- or 64-byte swizzle
                    uint8_t *piece = staging.next();
                    uint4 *row = reinterpret_cast<uint4 *>(piece) + lane * (DW_F32 ? 8 : 4);
                    if (DW_F32) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            row[j ^ (lane & 7)] = make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                                             __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            row[j ^ ((lane >> 1) & 3)] =
                                make_uint4(pack_16(v[8 * j], v[8 * j + 1], p.bf16), pack_16(v[8 * j + 2], v[8 * j + 3], p.bf16),
                                           pack_16(v[8 * j + 4], v[8 * j + 5], p.bf16), pack_16(v[8 * j + 6], v[8 * j + 7], p.bf16));
                    }
                    staging.store(&map_dw, piece, int(k0), int(n0), x.group);
                    continue;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    tile[lane * 8 + (j ^ (lane & 7))] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                __syncwarp();
                if (DW_F32) {
                    const int q = lane & 7;
                    const int64_t k = k0 + 4 * q;
                    float4 o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = 4 * i + (lane >> 3);
                        o[i] = tile[r * 8 + (q ^ (r & 7))];
                    }
                    float *dst = static_cast<float *>(p.dW) + int64_t(x.group) * p.stridedw + (n0 + (lane >> 3)) * p.lddw + k;
#pragma unroll
                    for (int i = 0; i < 8; ++i, dst += 4 * p.lddw) {
                        if (n0 + 4 * i + (lane >> 3) >= p.N) continue;
                        if (k + 4 <= p.K) {
                            *reinterpret_cast<float4 *>(dst) = o[i];
                        } else {
                            const float e[4] = {o[i].x, o[i].y, o[i].z, o[i].w};
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (k + j < p.K) dst[j] = e[j];
                        }
                    }
                } else {
                    // lane: 8 columns of rows 8 i + lane / 4, two staged pieces to one 16-byte store
                    const int q = lane & 3;
                    const int64_t k = k0 + 8 * q;
                    uint4 o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 8 * i + (lane >> 2);
                        const float4 a = tile[r * 8 + ((2 * q) ^ (r & 7))], b = tile[r * 8 + ((2 * q + 1) ^ (r & 7))];
                        o[i] = make_uint4(pack_16(a.x, a.y, p.bf16), pack_16(a.z, a.w, p.bf16), pack_16(b.x, b.y, p.bf16),
                                          pack_16(b.z, b.w, p.bf16));
                    }
                    uint16_t *dst = static_cast<uint16_t *>(p.dW) + int64_t(x.group) * p.stridedw + (n0 + (lane >> 2)) * p.lddw + k;
#pragma unroll
                    for (int i = 0; i < 4; ++i, dst += 8 * p.lddw) {
                        if (n0 + 8 * i + (lane >> 2) >= p.N) continue;
                        if (k + 8 <= p.K) {
                            *reinterpret_cast<uint4 *>(dst) = o[i];
                        } else {
                            const uint32_t e[4] = {o[i].x, o[i].y, o[i].z, o[i].w};
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (k + j < p.K) dst[j] = uint16_t(e[j / 2] >> (16 * (j & 1)));
                        }
                    }
                }
            }
            if (x.rows == 0) continue;
            if (++acc == 2) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        staging.finish();
    }
    tear_down(tmem);
}

// ------------------------------------------------------------------ host side
// Row-major 16-bit matrices (a stack of `count`, `stride` elements apart; count 0: one matrix, 2-D
// map), read in boxes of 64 columns x box_rows with the 128-byte swizzle.
bool make_map(CUtensorMap *map, const void *ptr, bool bf16, int64_t rows, int64_t cols, int64_t ld, int box_rows,
              int64_t count, int64_t stride)
{
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    const cuuint32_t rank = count > 0 ? 3 : 2;
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(count)};
    const cuuint64_t strides[2] = {cuuint64_t(ld) * 2, cuuint64_t(stride) * 2};
    const cuuint32_t box[3] = {64, cuuint32_t(box_rows), 1};
    const cuuint32_t steps[3] = {1, 1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, const_cast<void *>(ptr),
              dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Tiling {
    int cap, splits;
};
constexpr int kMostSplits = 8;

// Tokens of a tile: the multiple of 32 for which the average group's tiles take the least time in
// waves of all pairs.  A K slice of a tile of w tokens takes the longer of its MMAs and of its copies
// and hand-overs; measured with 64 groups of 512 rows, K = 4096, in SM cycles: 375 (w = 32), 431 (128),
// 532 (192), 698 (256, where the chip's power limit sets the clock).  A tile costs about 8 slices more
// than it has.  Where the tiles leave pairs idle, K may be split among them at the cost of one more
// kernel, about 6000 cycles and the partial sums' way through L2 (work for `most_splits` of them).
Tiling tiling_of(int64_t rows, int64_t groups, int64_t ftiles, int64_t num_kb, int pairs, int most_splits)
{
    if (rows < groups) groups = rows;
    const int64_t mean = (rows + groups - 1) / groups;
    Tiling best{256, 1};
    double least = 1e300;
    // GEMM_GB300_GROUPED_CAP=n (sweeps only): tiles of at most n tokens
    int only = 0;
    if (const char *e = std::getenv("GEMM_GB300_GROUPED_CAP"); e && std::atoi(e) >= 32 && std::atoi(e) <= 256)
        only = std::atoi(e) / 32 * 32;
    for (int cap = 256; cap >= 32; cap -= 32) {
        if (only != 0 && cap != only) continue;
        const int64_t tiles = (mean + cap - 1) / cap;
        const int64_t width = ((mean + tiles - 1) / tiles + 31) / 32 * 32;
        const int64_t units = groups * tiles * ftiles;
        const double mma = 2.73 * double(width), copies = 360.0 + 0.55 * double(width);
        for (int splits = 1; splits <= most_splits && (splits == 1 || (units * splits <= pairs && num_kb >= 4 * splits)); ++splits) {
            const int64_t waves = (units * splits + pairs - 1) / pairs;
            const int64_t slices = (num_kb + splits - 1) / splits + 8;
            double cost = double(waves * slices) * (mma > copies ? mma : copies);
            if (splits > 1) cost += 6000.0 + 0.002 * double(rows * ftiles * 256 * splits);
            if (cost < 0.98 * least) {
                least = cost;
                best = Tiling{cap, splits};
            }
        }
    }
    return best;
}

template <int W_MN, int EPI, bool Y_F32>
cudaError_t launch_linear_t(const DeviceInfo &dev, const GroupedArgs &a, Tiling tiling, cudaStream_t stream)
{
    static std::atomic<int> cache[64];
    auto *kernel = grouped_linear_kernel<W_MN, EPI, Y_F32>;
    const int pairs = resident_pairs(kernel, kThreads, kSmemBytes, dev.device, cache);
    unsigned int *status = device_status_word(dev.device);
    if (pairs <= 0 || status == nullptr) return cudaErrorInitializationError;
    const bool bf16 = a.type == GEMM_TYPE_BF16;
    const int64_t w_rows = a.opW == GEMM_OP_T ? (a.gated ? 2 * a.N : a.N) : a.K;
    const int64_t w_cols = a.opW == GEMM_OP_T ? a.K : a.N;
    const bool shared_w = a.groups == 1 || a.stridew == 0;
    CUtensorMap mw;
    TokenMaps mx;
    std::memset(&mw, 0, sizeof(mw));
    std::memset(&mx, 0, sizeof(mx));
    bool ok = make_map(&mw, a.W, bf16, w_rows, w_cols, a.ldw, W_MN || EPI == kGated ? 64 : 128, shared_w ? 1 : a.groups,
                       shared_w ? w_rows * a.ldw : a.stridew);
    for (int i = 0; ok && i < (a.rows != nullptr ? 1 : 4); ++i)
        ok = make_map(&mx.rows[i], a.X, bf16, a.x_rows, a.K, a.ldx, a.rows != nullptr ? 1 : 128 >> i, 0, 0);
    CUtensorMap mb;
    TokenMaps mi;
    std::memset(&mb, 0, sizeof(mb));
    std::memset(&mi, 0, sizeof(mi));
    if (EPI == kAdapted) {
        const InnerLayout in = inner_layout(a.y_rows, a.ad.requests, a.ad.rank, a.ad.parts);
        ok = ok && make_map(&mb, a.ad.b, bf16, a.N, a.ad.rank, a.ad.ldb, 128, a.ad.count, a.ad.count > 1 ? a.ad.strideb : a.N * a.ad.ldb);
        for (int i = 0; ok && i < 4; ++i)
            ok = make_map(&mi.rows[i], a.ad.inner, bf16, in.plane_rows * in.parts * in.blocks, 64, 64, 128 >> i, 0, 0);
    }
    if (!ok) return cudaErrorInvalidValue;
    const int features = EPI == kGated ? 128 : 256;
    LinearParams p{};
    p.offsets = a.offsets;
    p.groups = a.groups;
    p.shared_w = shared_w;
    p.y_rows = a.y_rows;
    p.x_rows = a.x_rows;
    p.N = a.N;
    p.ftiles = int((a.N + features - 1) / features);
    p.num_kb = int((a.K + 63) / 64);
    p.cap = tiling.cap;
    p.splits = tiling.splits;
    p.split_stride = a.ldy * a.y_rows;
    CUtensorMap my;
    std::memset(&my, 0, sizeof(my));
    p.y_tma = make_store_map(&my, a.Y, a.y_type, a.y_rows, a.N, a.ldy, p.splits, p.split_stride, false);
    p.rows = a.rows;
    p.Y = a.Y;
    p.ldy = a.ldy;
    p.bf16 = bf16;
    p.pre = a.pre;
    p.ldp = a.ldp;
    if (EPI == kAdapted) {
        const InnerLayout in = inner_layout(a.y_rows, a.ad.requests, a.ad.rank, a.ad.parts);
        p.segments = a.ad.segments;
        p.adapters = a.ad.adapters;
        p.requests = a.ad.requests;
        p.n_adapters = a.ad.count;
        p.rank = a.ad.rank;
        p.parts = in.parts;
        p.plane_rows = int(in.plane_rows);
        p.values = reinterpret_cast<const float *>(static_cast<const char *>(a.ad.inner) + in.values_at());
        p.b = a.ad.b;
        p.ldb = a.ad.ldb;
        p.strideb = a.ad.strideb;
    }
    p.status = status;
    test_hooks(p.timeout_ns, p.inject_stall);
    // no more pairs than there can be units, which are counted in 32 bits
    const int64_t most = ((a.y_rows < a.groups ? a.y_rows : a.groups) + a.y_rows / p.cap) * p.ftiles * p.splits;
    if (most >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    return launch_chained(kernel, dim3(unsigned(2 * (most < pairs ? most : pairs))), kThreads, kSmemBytes, 2, stream, mw, mx, mb,
                          mi, my, p);
}

template <int W_MN, int EPI> cudaError_t launch_linear(const DeviceInfo &dev, const GroupedArgs &a, cudaStream_t stream)
{
    const int features = EPI == kGated ? 128 : 256;
    const bool splittable = EPI == kAdapted && a.work != nullptr;
    const Tiling tiling = tiling_of(a.y_rows, a.groups, (a.N + features - 1) / features, (a.K + 63) / 64, dev.num_sms / 2,
                                    splittable ? kMostSplits : 1);
    if (splittable && tiling.splits > 1) {
        GroupedArgs b = a;  // the partial sums
        b.Y = a.work;
        b.y_type = GEMM_TYPE_F32;
        b.ldy = (a.N + 7) / 8 * 8;
        const cudaError_t e = launch_linear_t<W_MN, EPI, true>(dev, b, tiling, stream);
        if (e != cudaSuccess) return e;
        return launch_sum(a.y_type, a.y_rows, a.N, tiling.splits, static_cast<const float *>(b.Y), b.ldy, a.Y, a.ldy, stream);
    }
    return a.y_type == GEMM_TYPE_F32 ? launch_linear_t<W_MN, EPI, true>(dev, a, tiling, stream)
                                     : launch_linear_t<W_MN, EPI, false>(dev, a, tiling, stream);
}

}  // namespace

int64_t split_bytes(int64_t rows, int64_t N, int64_t K, int pairs)
{
    const Tiling t = tiling_of(rows, 1, (N + 255) / 256, (K + 63) / 64, pairs, kMostSplits);
    return t.splits > 1 ? t.splits * rows * ((N + 7) / 8 * 8) * 4 : 0;
}

cudaError_t launch_many_rows(const DeviceInfo &dev, const GroupedArgs &a, cudaStream_t stream)
{
    if (dev.smem_optin < size_t(kSmemBytes)) return cudaErrorInvalidDevice;
    if (a.opW == GEMM_OP_N) return launch_linear<1, kPlain>(dev, a, stream);
    if (a.gated) return launch_linear<0, kGated>(dev, a, stream);
    if (a.ad.b != nullptr) return launch_linear<0, kAdapted>(dev, a, stream);
    return launch_linear<0, kPlain>(dev, a, stream);
}

cudaError_t launch_weight_grad(const DeviceInfo &dev, const WeightGradArgs &a, cudaStream_t stream)
{
    static std::atomic<int> cache[2][64];
    if (dev.smem_optin < size_t(kSmemBytes)) return cudaErrorInvalidDevice;
    const bool f32 = a.dw_type == GEMM_TYPE_F32;
    auto *kernel = f32 ? grouped_grad_kernel<true> : grouped_grad_kernel<false>;
    const int pairs = resident_pairs(kernel, kGradThreads, kSmemBytes, dev.device, cache[f32]);
    unsigned int *status = device_status_word(dev.device);
    if (pairs <= 0 || status == nullptr) return cudaErrorInitializationError;
    const bool bf16 = a.type == GEMM_TYPE_BF16;
    CUtensorMap md, mx;
    std::memset(&md, 0, sizeof(md));
    std::memset(&mx, 0, sizeof(mx));
    // without positions no copy is made: the maps stay empty
    if (a.positions > 0 && (!make_map(&md, a.dY, bf16, a.positions, a.N, a.lddy, 64, 0, 0) ||
                            !make_map(&mx, a.X, bf16, a.positions, a.K, a.ldx, 64, 0, 0)))
        return cudaErrorInvalidValue;
    GradParams p{};
    p.offsets = a.offsets;
    p.groups = a.groups;
    p.positions = a.positions;
    p.N = a.N;
    p.K = a.K;
    p.ntiles = int((a.N + 255) / 256);
    p.ktiles = int((a.K + 255) / 256);
    p.dW = a.dW;
    p.lddw = a.lddw;
    p.stridedw = a.stridedw;
    CUtensorMap mw;
    std::memset(&mw, 0, sizeof(mw));
    p.dw_tma = make_store_map(&mw, a.dW, a.dw_type, a.N, a.K, a.lddw, a.groups, a.stridedw, true);
    p.bf16 = bf16;
    p.status = status;
    test_hooks(p.timeout_ns, p.inject_stall);
    const int64_t units = int64_t(a.groups) * p.ntiles * p.ktiles;
    if (units >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    return launch_chained(kernel, dim3(unsigned(2 * (units < pairs ? units : pairs))), kGradThreads, kSmemBytes, 2, stream, md, mx,
                          mw, p);
}

}  // namespace gemm
