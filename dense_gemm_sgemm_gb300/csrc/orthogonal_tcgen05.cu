// The products of an orthogonalised update's step, X' = (a + b A + c A^2) X with A = X X^T, on the tcgen05
// tensor cores (semantics: include/gemm_gb300.h):
//
//     gram     A = X X^T               held as its diagonal d (fp32) and the rest E (two fp16 parts)
//     square   B = b A + c A^2         likewise f and F
//     update   X' = (a + f) X + F X    two fp16 parts; the last step writes the result
//
// A result in bf16 takes one fp16 product each, with fp32 sums.  Rounding all of A and B to fp16 would lose
// too much: their diagonals dominate and change by up to 2^-12 of themselves.  So what multiplies a whole row
// or column stays out of the products: with A = d + E, A^2 = d^2 + (d_i + d_j) E + E E, and of B X the
// diagonal's part f X; a X and b A take both parts of X and E (22 bits).  The terms beside a product take the
// high part that the product takes: what is then missing of A^2 and B X is (A dE + dE A) and B dX, dE and dX
// the low parts, which vanish where A and B do; with both parts beside high products a rank-one G grew a second
// singular value (up to 4 * 10^-2 of the result's norm).  Over five steps of the usual coefficients this is off
// by 0.1 to 1.5 * 10^-3 of the result's norm (random, low-rank, rank-one, graded spectra, 256 rows and more),
// where rounding the result to bf16 is 1.7 * 10^-3; with the diagonals inside the products it is up to 2.6,
// with bf16 iterates 12 to 55 * 10^-3.
//
// Small matrices, whose roundings do not average out and whose products are short of work anyway, and results
// in fp16 or fp32 take three products of the parts (high high + high low + low high): 10^-4 at most, for
// rank-one matrices, 10^-6 for most.  They run as three times the K slices.
//
// A and B are symmetric: only tiles on and below the diagonal are computed and stored, which halves two of the
// three products.  What a product needs of the others it reads from the tile on the other side of the diagonal,
// turned: the tensor cores take either order of an operand, slice by slice.
//
// Two forms, as the GEMM's: two CTAs on neighbouring SMs per 256 x 256 tile (cta_group::2), or one CTA per
// 128 x 128 tile; persistent, two accumulators, so that a tile's epilogue runs beside the next one's MMAs.
// Every wait is bounded: when one expires the kernel raises the device's error word, stops all roles, waits
// (bounded) for its own copies and MMAs in flight, frees its TMEM and returns.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdlib>
#include <cstring>

#include "orthogonal_internal.h"
#include "tcgen05_ptx.cuh"
#include "tcgen05_roles.cuh"
#include "tensor_map.h"

namespace gemm {
namespace {

constexpr int kEpiWarps = 8, kThreads = 32 * (2 + kEpiWarps);
constexpr int kOperand = 128 * 128, kStage = 2 * kOperand, kStages = 5;  // bytes: 128 rows of 64 fp16 of either operand
constexpr int kEpi = kEpiWarps * 4096, kIn = kEpiWarps * 4096, kBars = 256;  // what the epilogue stores, and reads
constexpr int kSmemBytes = kStages * kStage + kEpi + kIn + kBars + 1024;
static_assert(kSmemBytes <= 227 * 1024, "one CTA per SM");
constexpr unsigned kFull = 0xffffffffu;
constexpr int kGram = 0, kSquare = 1, kUpdate = 2, kResult = 3, kResultTurned = 4;

struct StepParams {
    int64_t n, k, ldk, ldn;  // sides and rows of the work matrices
    int count, tiles_m, tiles_n, per, num_kb;  // tiles of a matrix, K slices of one product
    int products;            // 1, or 3 of the parts
    int shift_a, shift_b;    // of a symmetric operand, whose tiles (of 2^shift) above the diagonal are not stored; else 0
    int64_t part_x, part_e;  // elements from the high part to the low one
    const __half *x, *e;
    float *d, *f;
    const float *unit;  // NULL: 1
    float a, b, c;
    float from_acc;            // the accumulator times this is the product
    float from_x, from_e, to;  // what the parts in memory are multiplied by, and what is stored
    void *Y;
    int64_t ldy, stridey, y_rows, y_cols;
    int y_tma, y_bf16;
    unsigned int *status;
    uint64_t timeout_ns;
    int inject_stall;  // test hook: the producer never fills its first slice
};

// Box of a 4-D tensor map: columns within a block of 64, rows, blocks of columns, plane.
template <bool PAIR>
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2, int c3)
{
    if constexpr (PAIR)
        asm volatile("cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
                     "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
                     "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                     : "memory");
}

// Whether columns k .. of rows m .. of a symmetric operand stored in tiles on and below the diagonal lie above
// it: they are read as rows k .. of columns m .., turned (MN-major).  m: the first row of the product's tile, for
// both CTAs of a pair: where the operand's tiles are smaller, the second CTA's are then on the diagonal at most.
__device__ __forceinline__ bool above(int k, int m, int shift) { return shift != 0 && k >> shift > m >> shift; }

struct Smem {
    uint32_t ring, bar0;
    uint8_t *epi, *in;
    volatile uint32_t *tmem_slot;
    volatile int *abort_flag;
    __device__ __forceinline__ explicit Smem(uint8_t *raw)
    {
        const uint32_t r = smem_u32(raw), base = (r + 1023u) & ~1023u;
        uint8_t *p = raw + (base - r);
        ring = base;
        epi = p + kStages * kStage;
        in = epi + kEpi;
        uint8_t *bars = in + kIn;
        bar0 = smem_u32(bars);
        tmem_slot = reinterpret_cast<volatile uint32_t *>(bars + kBars - 16);
        abort_flag = reinterpret_cast<volatile int *>(bars + kBars - 8);
    }
    __device__ __forceinline__ uint32_t full(int s) const { return bar0 + 8u * s; }
    __device__ __forceinline__ uint32_t empty(int s) const { return bar0 + 8u * (kStages + s); }
    __device__ __forceinline__ uint32_t acc_full(int i) const { return bar0 + 8u * (2 * kStages + i); }
    __device__ __forceinline__ uint32_t acc_empty(int i) const { return bar0 + 8u * (2 * kStages + 2 + i); }
    __device__ __forceinline__ uint32_t fetched(int w) const { return bar0 + 8u * (2 * kStages + 4 + w); }
    __device__ __forceinline__ uint32_t drain() const { return bar0 + 8u * (2 * kStages + 4 + kEpiWarps); }
    __device__ __forceinline__ uint32_t a(int s) const { return ring + uint32_t(s * kStage); }
    __device__ __forceinline__ uint32_t b(int s) const { return a(s) + kOperand; }
};

// Unit u: a matrix and a tile of it; of the symmetric products the tiles on and below the diagonal.
struct Unit {
    int which, tm, tn;
};
template <bool SYMMETRIC> __device__ __forceinline__ Unit unit_of(const StepParams &p, int u)
{
    Unit x;
    x.which = u / p.per;
    const int t = u - x.which * p.per;
    if (SYMMETRIC) {
        int m = int((sqrtf(8.0f * float(t) + 1.0f) - 1.0f) * 0.5f);
        while (m * (m + 1) / 2 > t) --m;
        while ((m + 1) * (m + 2) / 2 <= t) ++m;
        x.tm = m;
        x.tn = t - m * (m + 1) / 2;
    } else {  // groups of eight tile rows share their columns of X in L2
        const int group = t / (8 * p.tiles_n), rows = min(8, p.tiles_m - 8 * group), r = t - group * 8 * p.tiles_n;
        x.tm = 8 * group + r % rows;
        x.tn = r / rows;
    }
    return x;
}

// The parts of 32 elements of a row, from a warp's two boxes of 32 rows in the 64-byte swizzle.
struct Parts {
    uint4 h[4], l[4];
    __device__ __forceinline__ void load(const uint8_t *in, int lane)
    {
        const uint4 *row = reinterpret_cast<const uint4 *>(in) + lane * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = row[i ^ ((lane >> 1) & 3)];
            l[i] = row[128 + (i ^ ((lane >> 1) & 3))];
        }
    }
    __device__ __forceinline__ float high(int i) const { return __half2float(reinterpret_cast<const __half *>(h)[i]); }
    __device__ __forceinline__ float low(int i) const { return __half2float(reinterpret_cast<const __half *>(l)[i]); }
};

// Stores 32 columns of a row as their fp16 parts, the low one too if it is wanted.
__device__ __forceinline__ void store_parts(Staging<false> &staging, float (&v)[32], const CUtensorMap *map, int m0, int n0, int high,
                                            int low, bool both)
{
    store_rows<false>(staging, v, map, true, nullptr, 0, m0, n0, 0, 0, false, high);
    if (both) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const float2 h = __half22float2(__floats2half2_rn(v[i], v[i + 1]));
            v[i] -= h.x;
            v[i + 1] -= h.y;
        }
        store_rows<false>(staging, v, map, true, nullptr, 0, m0, n0, 0, 0, false, low);
    }
}
// Moves the diagonal out of a 32 x 32 piece on it: this lane's element to `to`, zero in its place.
__device__ __forceinline__ void take_diagonal(float (&v)[32], int lane, float *to, bool row)
{
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (lane == i) {
            d = v[i];
            v[i] = 0.0f;
        }
    if (row) *to = d;
}

template <bool PAIR, int WHAT, bool F32>
__global__ void __launch_bounds__(kThreads, 1)
orthogonal_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                  const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_in,
                  const __grid_constant__ CUtensorMap map_turned, const __grid_constant__ StepParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const Smem sh(smem_raw);
    constexpr bool kSymmetric = WHAT <= kSquare, kTurnB = !kSymmetric;  // B = X is stored K x N
    constexpr int kTile = PAIR ? 256 : 128, kTmem = 2 * kTile, kHalf = kTile / 2;  // kHalf: columns of an epilogue warp
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(sh.full(s), 1);
            mbar_init(sh.empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sh.acc_full(i), 1);
            mbar_init(sh.acc_empty(i), (PAIR ? 2 : 1) * kEpiWarps);
        }
        for (int w = 0; w < kEpiWarps; ++w) mbar_init(sh.fetched(w), 1);
        mbar_init(sh.drain(), 1);
        *sh.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (PAIR) cluster_sync();
    if (warp == 1) tmem_alloc<PAIR>(smem_u32(const_cast<uint32_t *>(sh.tmem_slot)), kTmem);
    chain_wait();
    tc_fence_before();
    if (PAIR) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *sh.tmem_slot;
    const Watch watch{sh.abort_flag, p.status, p.timeout_ns};
    const int slices = p.num_kb * p.products;  // high high, high low, low high
    const int units = p.count * p.per, first = PAIR ? int(cluster_id_x()) : int(blockIdx.x),
              step = PAIR ? int(cluster_count_x()) : int(gridDim.x);
    Ring ring(kStages);
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;

    if (warp == 0) {
        // ---------------- producer, one lane: 128 rows of A, 128 rows (or columns of K x N) of B
        if (elect_one()) {
            tma_prefetch_desc(&map_a);
            tma_prefetch_desc(&map_b);
            const uint32_t full0 = PAIR ? map_to_rank(sh.full(0), 0) : sh.full(0);
            bool starve = p.inject_stall != 0;
            for (int u = first; ok && u < units; u += step) {
                const Unit x = unit_of<kSymmetric>(p, u);
                const int m0 = x.tm * kTile + int(rank) * 128, n0 = x.tn * kTile + int(rank) * 128;
                for (int product = 0; ok && product < p.products; ++product) {  // high high, high low, low high
                    const int plane_a = x.which + (product == 2 ? p.count : 0), plane_b = x.which + (product == 1 ? p.count : 0);
                    for (int k = 0; k < 64 * p.num_kb; k += 64) {
                        ok = watch.wait(sh.empty(ring.stage), ring.phase ^ 1u);
                        if (!ok) break;
                        if (rank == 0) mbar_expect_tx(sh.full(ring.stage), (PAIR ? 2 : 1) * kStage);
                        if (!starve) {
                            const uint32_t full = full0 + 8u * ring.stage, a = sh.a(ring.stage), b = sh.b(ring.stage);
                            if (above(k, x.tm * kTile, p.shift_a)) tma_load_4d<PAIR>(a, &map_turned, full, 0, k, m0 / 64, plane_a);
                            else if (PAIR) tma_load_3d_pair(a, &map_a, full, k, m0, plane_a);
                            else tma_load_3d(a, &map_a, full, k, m0, plane_a);
                            if (kTurnB) tma_load_4d<PAIR>(b, &map_b, full, 0, k, n0 / 64, plane_b);
                            else if (above(k, x.tn * kTile, p.shift_b)) tma_load_4d<PAIR>(b, &map_turned, full, 0, k, n0 / 64, plane_b);
                            else if (PAIR) tma_load_3d_pair(b, &map_b, full, k, n0, plane_b);
                            else tma_load_3d(b, &map_b, full, k, n0, plane_b);
                        }
                        starve = false;
                        ring.next();
                    }
                }
            }
            if (!ok) {  // copies in flight get time to land
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 2000000ull) {
                }
            } else {  // no commit is on its way to this CTA's barriers when it exits
                for (int i = 0; i < kStages; ++i) {
                    if (!watch.wait(sh.empty(ring.stage), ring.phase ^ 1u)) break;
                    ring.next();
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // ---------------- MMA issuer, one lane
            if (elect_one()) {
                // either operand by rows, or turned: its 64 k are rows of two blocks of 64 columns
                const uint64_t by_rows = smem_desc(sh.ring, 16, 1024), turned = smem_desc(sh.ring, kOperand / 2, 1024);
                const uint32_t idesc = make_idesc(0, 0, kTile, kTile);
                auto commit = [&](uint32_t bar) {
                    if (PAIR) commit_both(bar);
                    else umma_commit<false>(bar);
                };
                for (int u = first; ok && u < units; u += step) {
                    ok = watch.wait<true>(sh.acc_empty(acc), acc_phase ^ 1u);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + uint32_t(acc * kTile);
                    const Unit x = unit_of<kSymmetric>(p, u);
                    uint32_t more = 0u;
                    for (int i = 0, k = 0; i < slices; ++i, k = k + 64 == 64 * p.num_kb ? 0 : k + 64) {
                        ok = watch.wait(sh.full(ring.stage), ring.phase);
                        if (!ok) break;
                        tc_fence_after();
                        const bool turn_a = above(k, x.tm * kTile, p.shift_a), turn_b = kTurnB || above(k, x.tn * kTile, p.shift_b);
                        const uint64_t a = (turn_a ? turned : by_rows) + uint32_t(ring.stage * (kStage >> 4));
                        const uint64_t b = (turn_b ? turned : by_rows) + uint32_t(ring.stage * (kStage >> 4) + (kOperand >> 4));
                        const uint32_t step_a = (turn_a ? 2048 : 32) >> 4, step_b = (turn_b ? 2048 : 32) >> 4;
                        const uint32_t how = idesc | uint32_t(turn_a) << 15 | uint32_t(turn_b) << 16;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            umma_f16<PAIR>(d, a + q * step_a, b + q * step_b, how, more);
                            more = 1u;
                        }
                        commit(sh.empty(ring.stage));
                        ring.next();
                    }
                    if (!ok) break;
                    commit(sh.acc_full(acc));
                    acc ^= 1;
                    acc_phase ^= acc == 0 ? 1u : 0u;
                }
                if (!ok) {  // MMAs in flight finish before TMEM is released
                    umma_commit<PAIR>(sh.drain());
                    const volatile int no_abort = 0;
                    mbar_wait(sh.drain(), 0, &no_abort, 100000000ull);
                }
            }
        }
    } else {
        // ---------------- epilogue: rows 32 * quarter .. of this CTA's 128, half of the tile's columns
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        Staging<F32> staging(sh.epi + (warp - 2) * 4096, lane);
        const uint8_t *in = sh.in + (warp - 2) * 4096;
        uint32_t in_phase = 0;
        const uint32_t acc_empty0 = PAIR ? map_to_rank(sh.acc_empty(0), 0) : sh.acc_empty(0);
        for (int u = first; u < units; u += step) {
            const Unit x = unit_of<kSymmetric>(p, u);
            const int m0 = x.tm * kTile + int(rank) * 128 + quarter * 32, m = m0 + lane;
            const bool row = m < p.n;
            // what the epilogue reads is on its way during the products and the stores before it
            Parts old;
            auto inside = [&](int n0) { return m0 < p.n && n0 < (kSymmetric ? p.n : p.k); };
            auto fetch = [&](int n0) {
                if (WHAT == kGram || !inside(n0)) return;
                __syncwarp();  // the boxes before have been read
                if (lane == 0) {
                    const uint32_t dst = smem_u32(in), bar = sh.fetched(warp - 2);
                    mbar_expect_tx(bar, 4096);
                    tma_load_3d(dst, &map_in, bar, n0, m0, x.which);
                    tma_load_3d(dst + 2048, &map_in, bar, n0, m0, p.count + x.which);
                }
            };
            fetch(x.tn * kTile + half * kHalf);
            const float unit = p.unit != nullptr ? __ldg(p.unit + x.which) : 1.0f;
            float mine = 0.0f;  // d or f of this row
            if (WHAT == kSquare && row) mine = __ldcg(p.d + x.which * p.ldn + m);
            if (WHAT >= kUpdate && row) mine = __ldcg(p.f + x.which * p.ldn + m);
            ok = __all_sync(kFull, watch.wait(sh.acc_full(acc), acc_phase));
            if (!ok) break;
            tc_fence_after();
            const uint32_t taddr = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(acc * kTile + half * kHalf);
            const float scale = WHAT == kGram ? p.from_acc * unit * unit : WHAT == kSquare ? p.from_acc : p.from_acc * unit;
            const bool three = p.products == 3;
            const float from_x = p.from_x * unit, high = (p.a + mine) * from_x, low = three ? high : p.a * from_x;  // kUpdate
#pragma unroll 1
            for (int c = 0; c < kHalf; c += 32) {
                const int n0 = x.tn * kTile + half * kHalf + c;
                const bool wanted = inside(n0);
                float v[32];
                __syncwarp();
                tmem_ld_32(taddr + c, v);
                if (c + 32 >= kHalf) release_accumulator(acc_empty0 + 8u * acc, lane);
                if (!wanted) continue;
                if (WHAT != kGram) {
                    ok = __all_sync(kFull, watch.wait(sh.fetched(warp - 2), in_phase));
                    if (!ok) break;
                    in_phase ^= 1u;
                    old.load(in, lane);
                }
                if constexpr (WHAT == kGram) {
                    if (n0 == m0) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] *= scale;
                        take_diagonal(v, lane, p.d + x.which * p.ldn + m, row);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] *= p.to;
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = v[i] * scale * p.to;
                    }
                    store_parts(staging, v, &map_out, m0, n0, x.which, p.count + x.which, true);
                } else if constexpr (WHAT == kSquare) {
                    const float others = n0 + lane < p.n ? __ldcg(p.d + x.which * p.ldn + n0 + lane) : 0.0f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        // of A: E here, d on the diagonal, where E is 0; of A^2: (d_i + d_j) E + E E, d^2 + E E
                        const float hi = old.high(i) * p.from_e, e = fmaf(old.low(i), p.from_e, hi);
                        const float square = fmaf(three ? e : hi, mine + __shfl_sync(kFull, others, i), v[i] * scale);
                        v[i] = fmaf(p.b, e, p.c * square);
                    }
                    if (n0 == m0) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (lane == i) v[i] += fmaf(p.b, mine, p.c * mine * mine);
                        take_diagonal(v, lane, p.f + x.which * p.ldn + m, row);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] *= p.to;
                    if (c + 32 < kHalf) fetch(n0 + 32);
                    store_parts(staging, v, &map_out, m0, n0, x.which, p.count + x.which, three);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = fmaf(high, old.high(i), fmaf(low, old.low(i), v[i] * scale)) * p.to;
                    if (c + 32 < kHalf) fetch(n0 + 32);
                    if constexpr (WHAT == kUpdate) {
                        store_parts(staging, v, &map_out, m0, n0, x.which, p.count + x.which, true);
                    } else {
                        uint8_t *Y = static_cast<uint8_t *>(p.Y) + x.which * p.stridey * (F32 ? 4 : 2);
                        constexpr bool kTurned = WHAT == kResultTurned;
                        store_rows<F32, kTurned>(staging, v, &map_out, p.y_tma, Y, p.ldy, kTurned ? n0 : m0, kTurned ? m0 : n0, p.y_rows,
                                                 p.y_cols, p.y_bf16, x.which);
                    }
                }
            }
            if (!ok) break;
            acc ^= 1;
            acc_phase ^= acc == 0 ? 1u : 0u;
        }
        staging.finish();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // neither CTA leaves or frees TMEM while the other may still use it
    tc_fence_after();
    if (warp == 1) tmem_free<PAIR>(tmem, kTmem);
}

// ------------------------------------------------------------------ host side
// fp16 matrices (a stack of `count`) read in boxes of 64 columns x box_rows with the 128-byte swizzle.
bool make_map16(CUtensorMap *map, const void *ptr, int64_t rows, int64_t cols, int64_t ld, int64_t count, int box_rows)
{
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(count)};
    const cuuint64_t strides[2] = {cuuint64_t(ld) * 2, cuuint64_t(ld) * cuuint64_t(rows) * 2};
    const cuuint32_t box[3] = {64, cuuint32_t(box_rows), 1}, steps[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same matrices read as K x N operands, two blocks of 64 columns x 64 rows a box.  Columns between the
// matrix's end and its padded rows' end are read as they are: they only meet columns of the result beyond it.
bool make_map_columns(CUtensorMap *map, const void *ptr, int64_t rows, int64_t ld, int64_t count)
{
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    const cuuint64_t dims[4] = {64, cuuint64_t(rows), cuuint64_t(ld / 64), cuuint64_t(count)};
    const cuuint64_t strides[3] = {cuuint64_t(ld) * 2, 128, cuuint64_t(ld) * cuuint64_t(rows) * 2};
    const cuuint32_t box[4] = {64, 64, 2, 1}, steps[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(ptr), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pairs of SMs where the tiles' waves cost less.  A slice of 64 k takes a pair 560 SM cycles, a single CTA
// 330; a tile costs about 8 slices more than it has.
bool pairs_pay(const DeviceInfo &dev, int64_t count, int64_t m, int64_t n, bool symmetric, int64_t slices)
{
    auto tiles = [&](int64_t t) {
        const int64_t i = (m + t - 1) / t, j = (n + t - 1) / t;
        return count * (symmetric ? i * (i + 1) / 2 : i * j);
    };
    const int64_t pairs = dev.num_sms / 2;
    const double two = double((tiles(256) + pairs - 1) / pairs) * double(slices + 8) * 560.0;
    const double one = double((tiles(128) + dev.num_sms - 1) / dev.num_sms) * double(slices + 8) * 330.0;
    // GEMM_GB300_ORTHOGONAL_PAIR=0|1 (tests and sweeps): never, or always
    if (const char *e = std::getenv("GEMM_GB300_ORTHOGONAL_PAIR"); e && (*e == '0' || *e == '1')) return *e == '1';
    return two < one;
}

template <bool PAIR, int WHAT, bool F32>
cudaError_t launch_product(const DeviceInfo &dev, const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &out, const CUtensorMap &in, const CUtensorMap &turned, StepParams p,
                           int64_t columns, cudaStream_t stream)
{
    constexpr int kTile = PAIR ? 256 : 128;
    auto *kernel = orthogonal_kernel<PAIR, WHAT, F32>;
    int room;
    if (PAIR) {
        static std::atomic<int> cache[64];
        room = resident_pairs(kernel, kThreads, kSmemBytes, dev.device, cache);
        if (room <= 0) return cudaErrorInitializationError;
    } else {
        const cudaError_t e = allow_smem_once(kernel, kSmemBytes);
        if (e != cudaSuccess) return e;
        room = dev.num_sms;
    }
    p.tiles_m = int((p.n + kTile - 1) / kTile);
    p.tiles_n = int((columns + kTile - 1) / kTile);
    const int64_t per = WHAT <= kSquare ? int64_t(p.tiles_m) * (p.tiles_m + 1) / 2 : int64_t(p.tiles_m) * p.tiles_n;
    if (per * p.count >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    p.per = int(per);
    const int64_t units = per * p.count, grid = (units < room ? units : room) * (PAIR ? 2 : 1);
    return launch_chained(kernel, dim3(unsigned(grid)), kThreads, kSmemBytes, PAIR ? 2 : 1, stream, a, b, out, in, turned, p);
}
template <int WHAT, bool F32 = false>
cudaError_t launch_product(const DeviceInfo &dev, const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &out, const CUtensorMap &in, const CUtensorMap &turned, const StepParams &p, bool pairs,
                           int64_t columns, cudaStream_t stream)
{
    return pairs ? launch_product<true, WHAT, F32>(dev, a, b, out, in, turned, p, columns, stream)
                 : launch_product<false, WHAT, F32>(dev, a, b, out, in, turned, p, columns, stream);
}

}  // namespace

cudaError_t launch_orthogonal_step(const DeviceInfo &dev, const OrthogonalArgs &a, const OrthogonalLayout &l, const OrthogonalStep &s,
                                   int from, cudaStream_t stream)
{
    unsigned int *status = device_status_word(dev.device);
    if (status == nullptr || dev.smem_optin < size_t(kSmemBytes)) return cudaErrorInitializationError;
    char *w = static_cast<char *>(a.work);
    StepParams p{};
    p.n = l.n;
    p.k = l.k;
    p.ldk = l.ldk;
    p.ldn = l.ldn;
    p.count = int(l.count);
    p.part_x = l.count * l.n * l.ldk;
    p.part_e = l.count * l.n * l.ldn;
    p.x = reinterpret_cast<const __half *>(w + l.x[from]);
    p.e = reinterpret_cast<const __half *>(w + l.e);
    p.d = reinterpret_cast<float *>(w + l.dd);
    p.f = reinterpret_cast<float *>(w + l.df);
    p.products = s.products;
    p.a = s.a;
    p.b = s.b;
    p.c = s.c;
    p.status = status;
    test_hooks(p.timeout_ns, p.inject_stall);
    const float *unit = s.first ? reinterpret_cast<const float *>(w + l.unit) : nullptr;
    CUtensorMap x_rows, x_cols, e_rows, e_cols, f_rows, f_cols, e_out, f_out, x_in, x_out, y_out;
    std::memset(&y_out, 0, sizeof(y_out));
    if (!make_map16(&x_rows, p.x, l.n, l.k, l.ldk, 2 * l.count, 128) || !make_map_columns(&x_cols, p.x, l.n, l.ldk, 2 * l.count) || !make_map_columns(&e_cols, p.e, l.n, l.ldn, 2 * l.count) ||
        !make_map_columns(&f_cols, w + l.f, l.n, l.ldn, 2 * l.count) ||
        !make_map16(&e_rows, p.e, l.n, l.n, l.ldn, 2 * l.count, 128) || !make_map16(&f_rows, w + l.f, l.n, l.n, l.ldn, 2 * l.count, 128) ||
        !make_store_map(&e_out, w + l.e, GEMM_TYPE_F16, l.n, l.ldn, l.ldn, 2 * l.count, l.n * l.ldn, true) ||
        !make_store_map(&f_out, w + l.f, GEMM_TYPE_F16, l.n, l.ldn, l.ldn, 2 * l.count, l.n * l.ldn, true) ||
        !make_store_map(&x_in, w + l.x[from], GEMM_TYPE_F16, l.n, l.ldk, l.ldk, 2 * l.count, l.n * l.ldk, true) ||
        !make_store_map(&x_out, w + l.x[from ^ 1], GEMM_TYPE_F16, l.n, l.ldk, l.ldk, 2 * l.count, l.n * l.ldk, true))
        return cudaErrorInvalidValue;

    StepParams gram = p;
    gram.num_kb = int((l.k + 63) / 64);
    gram.unit = unit;
    gram.from_acc = 1.0f / (s.x_scale * s.x_scale);
    gram.to = s.e_scale;
    // the square's tiles are the Gram matrix's: what it reads beside them must be stored
    const bool pairs = pairs_pay(dev, l.count, l.n, l.n, true, gram.num_kb * p.products);
    cudaError_t e = launch_product<kGram>(dev, x_rows, x_rows, e_out, x_in, x_cols, gram, pairs, l.n, stream);
    if (e != cudaSuccess) return e;

    StepParams square = p;
    square.num_kb = int((l.n + 63) / 64);
    square.from_e = 1.0f / s.e_scale;
    square.from_acc = square.from_e * square.from_e;
    square.to = s.f_scale;
    square.shift_a = square.shift_b = pairs ? 8 : 7;
    e = launch_product<kSquare>(dev, e_rows, e_rows, f_out, e_out, e_cols, square, pairs, l.n, stream);
    if (e != cudaSuccess) return e;

    StepParams update = p;
    update.num_kb = square.num_kb;
    update.unit = unit;
    update.from_x = 1.0f / s.x_scale;
    update.from_acc = update.from_x / s.f_scale;
    update.to = s.last ? 1.0f : s.next_scale;
    update.shift_a = square.shift_a;
    const bool wide = pairs_pay(dev, l.count, l.n, l.k, false, update.num_kb * p.products);
    if (!s.last) return launch_product<kUpdate>(dev, f_rows, x_cols, x_out, x_in, f_cols, update, wide, l.k, stream);
    update.Y = a.Y;
    update.ldy = a.ldy;
    update.stridey = a.stridey;
    update.y_rows = a.rows;
    update.y_cols = a.cols;
    update.y_tma = make_store_map(&y_out, a.Y, a.y_type, a.rows, a.cols, a.ldy, l.count, a.stridey, true);
    update.y_bf16 = a.y_type == GEMM_TYPE_BF16;
    if (a.y_type == GEMM_TYPE_F32)
        return a.rows > a.cols ? launch_product<kResultTurned, true>(dev, f_rows, x_cols, y_out, x_in, f_cols, update, wide, l.k, stream)
                               : launch_product<kResult, true>(dev, f_rows, x_cols, y_out, x_in, f_cols, update, wide, l.k, stream);
    return a.rows > a.cols ? launch_product<kResultTurned>(dev, f_rows, x_cols, y_out, x_in, f_cols, update, wide, l.k, stream)
                           : launch_product<kResult>(dev, f_rows, x_cols, y_out, x_in, f_cols, update, wide, l.k, stream);
}

}  // namespace gemm
