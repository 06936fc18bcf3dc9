// The products of an orthogonalised update's step, X' = (a + b A + c A^2) X with A = X X^T, on the tcgen05
// tensor cores (semantics: include/gemm_gb300.h):
//
//     gram     A = X X^T               held as its diagonal d (fp32) and the rest E (two fp16 parts)
//     square   B = b A + c A^2         likewise f and F
//     update   X' = (a + f) X + F X    two fp16 parts; the last step writes the result
//
// Each is three products of the parts (high low + low high + high high), as three times the K slices.  One fp16 product
// of the high parts would not do even for a bf16 result: where elements are equal in magnitude their roundings are
// equal too and do not average out, and the steps multiply them (a constant 512 x 512 came to 1.3 * 10^-2 of the
// result's norm, a matrix of equal rows to 6 * 10^-3, where rounding the result to bf16 is 1.7 * 10^-3 at most).  Nor
// would two, with one operand's low part left out.  The small products come first: the tensor cores' fp32 sums round
// towards zero at every 16 k, and after the large product each of their additions would lose a step of the whole sum
// (equal rows, 4096 x 4096: 2.1 * 10^-3, now 3 * 10^-4; the formula in fp32 3.3 * 10^-4).  What is left is 10^-6 for
// most matrices of 1000 rows, 3 * 10^-5 for 4096, and up to 1.5 * 10^-3 for 4096 x 4096 of rank two.
//
// What multiplies a whole row or column stays out of the products: with A = d + E, A^2 = d^2 + (d_i + d_j) E + E E, and
// of B X the diagonal's part f X, so the products' roundings are those of the rest, and d and f are held in fp32.
//
// A and B are symmetric: only tiles on and below the diagonal are computed and stored, which halves two of the
// three products.  What a product needs of the others it reads from the tile on the other side of the diagonal,
// turned: the tensor cores take either order of an operand, slice by slice.  Within a tile on the diagonal the 32 x 32
// above it are stored turned too, from those below: with three products an element and its mirror image are summed
// in different orders, and of the two one is kept.  So it makes no difference which of them a form reads, and a
// result is the same to the bit in every form, and with it alone and in any stack.
//
// Four forms: two CTAs on neighbouring SMs per tile of 256 x 256 or 256 x 128 (cta_group::2), or one CTA per
// 128 x 128 or 128 x 64 tile; persistent, two accumulators, so that a tile's epilogue runs beside the next one's MMAs.
//
// What bounds them (GB300; the three products of a step, each alone).  4096 x 4096: 126, 126 and 250 us, 1.65 to 1.74
// PFLOP/s, the tensor pipe 88 to 94% active; one after another the power limit takes 10% more.  2048 x 4096: 44, 30
// and 67 us: 72 tiles of 256 x 128 in one wave, whose epilogue nothing hides, and 128 of 256 x 256 on 76 pairs.
// 256 x 512: about 6 us each in the chain, of which the MMAs are 1: a launch's hand-over (1.4 to 2.1), the first
// copies, one epilogue and its stores.
//
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

constexpr int kEpiWarps = 8, kFirst = 3, kThreads = 32 * (kFirst + kEpiWarps);  // kFirst: the first epilogue warp
constexpr int kOperandA = 128 * 128;  // bytes: 128 rows of 64 fp16
constexpr int kEpi = kEpiWarps * 4096, kIn = kEpiWarps * 4096, kBars = 256;  // what the epilogue stores, and reads
// The forms: a CTA's 128 x 128, a pair's 256 x 128, a pair's 256 x 256, a CTA's 128 x 64.
constexpr bool is_pair(int form) { return form == 1 || form == 2; }
constexpr int tile_m(int form) { return is_pair(form) ? 256 : 128; }
constexpr int tile_n(int form) { return form == 2 ? 256 : form == 3 ? 64 : 128; }
template <int FORM> struct Shape {
    static constexpr bool kPair = is_pair(FORM);
    static constexpr int kM = tile_m(FORM), kN = tile_n(FORM), kRowsB = kPair ? kN / 2 : kN;  // rows of B a CTA holds
    static constexpr int kStage = kOperandA + kRowsB * 128, kStages = FORM & 1 ? 6 : 5;
    static constexpr int kBytes = kStages * kStage + kEpi + kIn + kBars + 1024;
    static_assert(kBytes <= 227 * 1024, "one CTA per SM");
};
constexpr int kMostBytes = Shape<2>::kBytes;
constexpr unsigned kFull = 0xffffffffu;
constexpr int kProducts = 3;  // of the parts
constexpr int kGram = 0, kSquare = 1, kUpdate = 2, kResult = 3, kResultTurned = 4;

struct StepParams {
    int64_t n, k, ldn;       // sides, and distance of two matrices' diagonals
    int count, tiles_m, tiles_n, per, num_kb;  // tiles of a matrix, K slices of one product
    int shift_a, shift_b;    // of a symmetric operand, whose tiles (of 2^shift) above the diagonal are not stored; else 0
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

template <int FORM> struct Smem {
    static constexpr int kStages = Shape<FORM>::kStages, kStage = Shape<FORM>::kStage;
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
    __device__ __forceinline__ uint32_t b(int s) const { return a(s) + kOperandA; }
};

// Unit u: a matrix and a tile of it; of the symmetric products the tiles on and below the diagonal, of which a
// row of tiles has W = kM / kN more than the one before (the last columns of the last row may lie outside).
struct Unit {
    int which, tm, tn;
};
template <bool SYMMETRIC, int W> __device__ __forceinline__ Unit unit_of(const StepParams &p, int u)
{
    Unit x;
    x.which = u / p.per;
    const int t = u - x.which * p.per;
    if (SYMMETRIC) {
        const float s = float(t) / W;
        int m = int((sqrtf(8.0f * s + 1.0f) - 1.0f) * 0.5f);
        while (W * (m * (m + 1) / 2) > t) --m;
        while (W * ((m + 1) * (m + 2) / 2) <= t) ++m;
        x.tm = m;
        x.tn = t - W * (m * (m + 1) / 2);
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

// Stores 32 columns of a row as their fp16 parts; turned: on the other side of the diagonal as well.
__device__ __forceinline__ void store_parts(Staging<false> &staging, float (&v)[32], const CUtensorMap *map, int m0, int n0, int high,
                                            int low, bool turned)
{
    store_rows<false>(staging, v, map, true, nullptr, 0, m0, n0, 0, 0, false, high);
    if (turned) store_rows<false, true>(staging, v, map, true, nullptr, 0, n0, m0, 0, 0, false, high);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        const float2 h = __half22float2(__floats2half2_rn(v[i], v[i + 1]));
        v[i] -= h.x;
        v[i + 1] -= h.y;
    }
    store_rows<false>(staging, v, map, true, nullptr, 0, m0, n0, 0, 0, false, low);
    if (turned) store_rows<false, true>(staging, v, map, true, nullptr, 0, n0, m0, 0, 0, false, low);
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
// A 32 x 32 piece on the diagonal: what is above it, from below it.  tile: 4 KB of the warp's own.
__device__ __forceinline__ void mirror(float (&v)[32], int lane, float *tile)
{
#pragma unroll
    for (int i = 0; i < 32; ++i) tile[lane * 32 + (i ^ lane)] = v[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (i > lane) v[i] = tile[i * 32 + (lane ^ i)];
    __syncwarp();
}

template <int FORM, int WHAT, bool F32>
__global__ void __launch_bounds__(kThreads, 1)
orthogonal_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                  const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_in,
                  const __grid_constant__ CUtensorMap turned_a, const __grid_constant__ CUtensorMap turned_b,
                  const __grid_constant__ StepParams p)
{
    extern __shared__ uint8_t smem_raw[];
    using S = Shape<FORM>;
    const Smem<FORM> sh(smem_raw);
    constexpr bool PAIR = S::kPair;
    constexpr int kStage = S::kStage, kStages = S::kStages;
    constexpr bool kSymmetric = WHAT <= kSquare, kTurnB = !kSymmetric;  // B = X is stored K x N
    constexpr int kTmem = 2 * S::kN, kHalf = S::kN / 2;  // kHalf: columns of an epilogue warp
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
    const int slices = p.num_kb * kProducts;
    const int units = p.count * p.per, first = PAIR ? int(cluster_id_x()) : int(blockIdx.x),
              step = PAIR ? int(cluster_count_x()) : int(gridDim.x);
    Ring ring(kStages);
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;

    if (warp == 0 || warp == 2) {
        // ---------------- producers, one lane each: 128 rows of A; rows of B (or columns of K x N).  (One for both
        // takes longer to issue a slice's copies than the tensor cores to multiply it.)
        if (elect_one()) {
            const bool of_a = warp == 0;
            tma_prefetch_desc(of_a ? &map_a : &map_b);
            const uint32_t full0 = PAIR ? map_to_rank(sh.full(0), 0) : sh.full(0);
            bool starve = p.inject_stall != 0;
            for (int u = first; ok && u < units; u += step) {
                const Unit x = unit_of<kSymmetric, S::kM / S::kN>(p, u);
                const int row = of_a ? x.tm * S::kM + int(rank) * 128 : x.tn * S::kN + int(rank) * S::kRowsB;
                const int of_tile = of_a ? x.tm * S::kM : x.tn * S::kN, shift = of_a ? p.shift_a : p.shift_b;
                for (int product = 0; ok && product < kProducts; ++product) {  // high low, low high, high high
                    const int plane = x.which + (product == (of_a ? 1 : 0) ? p.count : 0);
                    for (int k = 0; k < 64 * p.num_kb; k += 64) {
                        ok = watch.wait(sh.empty(ring.stage), ring.phase ^ 1u);
                        if (!ok) break;
                        if (of_a && rank == 0) mbar_expect_tx(sh.full(ring.stage), (PAIR ? 2 : 1) * kStage);
                        if (!starve) {
                            const uint32_t full = full0 + 8u * ring.stage, dst = of_a ? sh.a(ring.stage) : sh.b(ring.stage);
                            if ((!of_a && kTurnB) || above(k, of_tile, shift))
                                tma_load_4d<PAIR>(dst, of_a ? &turned_a : kTurnB ? &map_b : &turned_b, full, 0, k, row / 64, plane);
                            else if (PAIR) tma_load_3d_pair(dst, of_a ? &map_a : &map_b, full, k, row, plane);
                            else tma_load_3d(dst, of_a ? &map_a : &map_b, full, k, row, plane);
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
            } else if (of_a) {  // no commit is on its way to this CTA's barriers when it exits
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
                const uint64_t by_rows = smem_desc(sh.ring, 16, 1024), turned = smem_desc(sh.ring, kOperandA / 2, 1024);
                const uint32_t idesc = make_idesc(0, 0, S::kN, S::kM);
                auto commit = [&](uint32_t bar) {
                    if (PAIR) commit_both(bar);
                    else umma_commit<false>(bar);
                };
                for (int u = first; ok && u < units; u += step) {
                    ok = watch.wait<true>(sh.acc_empty(acc), acc_phase ^ 1u);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + uint32_t(acc * S::kN);
                    const Unit x = unit_of<kSymmetric, S::kM / S::kN>(p, u);
                    uint32_t more = 0u;
                    for (int i = 0, k = 0; i < slices; ++i, k = k + 64 == 64 * p.num_kb ? 0 : k + 64) {
                        ok = watch.wait(sh.full(ring.stage), ring.phase);
                        if (!ok) break;
                        tc_fence_after();
                        const bool turn_a = above(k, x.tm * S::kM, p.shift_a), turn_b = kTurnB || above(k, x.tn * S::kN, p.shift_b);
                        const uint64_t a = (turn_a ? turned : by_rows) + uint32_t(ring.stage * (kStage >> 4));
                        const uint64_t b = (turn_b ? turned : by_rows) + uint32_t(ring.stage * (kStage >> 4) + (kOperandA >> 4));
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
        const int quarter = warp & 3, half = (warp - kFirst) >> 2;
        Staging<F32> staging(sh.epi + (warp - kFirst) * 4096, lane);
        const uint8_t *in = sh.in + (warp - kFirst) * 4096;
        uint32_t in_phase = 0;
        const uint32_t acc_empty0 = PAIR ? map_to_rank(sh.acc_empty(0), 0) : sh.acc_empty(0);
        for (int u = first; u < units; u += step) {
            const Unit x = unit_of<kSymmetric, S::kM / S::kN>(p, u);
            const int m0 = x.tm * S::kM + int(rank) * 128 + quarter * 32, m = m0 + lane;
            const bool row = m < p.n;
            // what the epilogue reads is on its way during the products and the stores before it
            Parts old;
            const int columns = x.tn * S::kN + half * kHalf;
            auto inside = [&](int n0) { return m0 < p.n && n0 < (kSymmetric ? min(p.n, int64_t(m0) + 32) : p.k); };
            auto fetch = [&](int n0) {
                if (WHAT == kGram || !inside(n0)) return;
                __syncwarp();  // the boxes before have been read
                if (lane == 0) {
                    const uint32_t dst = smem_u32(in), bar = sh.fetched(warp - kFirst);
                    mbar_expect_tx(bar, 4096);
                    tma_load_3d(dst, &map_in, bar, n0, m0, x.which);
                    tma_load_3d(dst + 2048, &map_in, bar, n0, m0, p.count + x.which);
                }
            };
            fetch(columns);
            const float unit = p.unit != nullptr ? load_now(p.unit + x.which) : 1.0f;
            float mine = 0.0f;  // d or f of this row
            if (WHAT == kSquare && row) mine = __ldcg(p.d + x.which * p.ldn + m);
            if (WHAT >= kUpdate && row) mine = __ldcg(p.f + x.which * p.ldn + m);
            ok = __all_sync(kFull, watch.wait(sh.acc_full(acc), acc_phase));
            if (!ok) break;
            tc_fence_after();
            const uint32_t taddr = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(acc * S::kN + half * kHalf);
            const float scale = WHAT == kGram ? p.from_acc * unit * unit : WHAT == kSquare ? p.from_acc : p.from_acc * unit;
            const float from_x = (p.a + mine) * (p.from_x * unit);  // kUpdate
#pragma unroll 1
            for (int c = 0; c < kHalf; c += 32) {
                const int n0 = columns + c;
                const bool wanted = inside(n0), under = n0 < m0 && n0 / S::kM == m0 / S::kM;  // under the diagonal, on its tile
                float v[32];
                __syncwarp();
                tmem_ld_32(taddr + c, v);
                if (c + 32 >= kHalf) release_accumulator(acc_empty0 + 8u * acc, lane);
                if (!wanted) continue;
                if (WHAT != kGram) {
                    ok = __all_sync(kFull, watch.wait(sh.fetched(warp - kFirst), in_phase));
                    if (!ok) break;
                    in_phase ^= 1u;
                    old.load(in, lane);
                }
                if constexpr (WHAT == kGram) {
                    if (n0 == m0) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] *= scale;
                        take_diagonal(v, lane, p.d + x.which * p.ldn + m, row);
                        mirror(v, lane, reinterpret_cast<float *>(staging.all()));
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] *= p.to;
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = v[i] * scale * p.to;
                    }
                    store_parts(staging, v, &map_out, m0, n0, x.which, p.count + x.which, under);
                } else if constexpr (WHAT == kSquare) {
                    const float others = n0 + lane < p.n ? __ldcg(p.d + x.which * p.ldn + n0 + lane) : 0.0f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        // of A: E here, d on the diagonal, where E is 0; of A^2: (d_i + d_j) E + E E, d^2 + E E
                        const float e = (old.high(i) + old.low(i)) * p.from_e;
                        const float square = fmaf(e, mine + __shfl_sync(kFull, others, i), v[i] * scale);
                        v[i] = fmaf(p.b, e, p.c * square);
                    }
                    if (n0 == m0) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (lane == i) v[i] += fmaf(p.b, mine, p.c * mine * mine);
                        take_diagonal(v, lane, p.f + x.which * p.ldn + m, row);
                        mirror(v, lane, reinterpret_cast<float *>(staging.all()));
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] *= p.to;
                    if (c + 32 < kHalf) fetch(n0 + 32);
                    store_parts(staging, v, &map_out, m0, n0, x.which, p.count + x.which, under);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = fmaf(from_x, old.high(i) + old.low(i), v[i] * scale) * p.to;
                    if (c + 32 < kHalf) fetch(n0 + 32);
                    if constexpr (WHAT == kUpdate) {
                        store_parts(staging, v, &map_out, m0, n0, x.which, p.count + x.which, false);
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
// The same matrices read as K x N operands, `blocks` blocks of 64 columns x 64 rows a box.  Columns between the
// matrix's end and its padded rows' end are read as they are: they only meet columns of the result beyond it.
bool make_map_columns(CUtensorMap *map, const void *ptr, int64_t rows, int64_t ld, int64_t count, int blocks)
{
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    const cuuint64_t dims[4] = {64, cuuint64_t(rows), cuuint64_t(ld / 64), cuuint64_t(count)};
    const cuuint64_t strides[3] = {cuuint64_t(ld) * 2, 128, cuuint64_t(ld) * cuuint64_t(rows) * 2};
    const cuuint32_t box[4] = {64, 64, cuuint32_t(blocks), 1}, steps[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(ptr), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int rows_b(int form) { return form & 1 ? 64 : 128; }

// The form whose waves of tiles cost least: a tile takes `slice` SM cycles a slice of 64 k and as much for `more`
// slices beyond its own.  The symmetric products take one form, for the `slices` of both (other: the square's).
// Fitted to 29 shapes, from 64 x 64 to 4096 x 4096 and stacks of up to 60, each in all 16 pairs of forms; of 17 of them the
// ones taken are on average 0.8% slower than the fastest pair.  (Whole calls: 256 x 512 104 us with 128 x 64, 128 with
// 128 x 128, 137 and 197 with pairs; 2048 x 4096 with 256 x 256 and the symmetric ones in 256 x 128 657 us, the other
// forms throughout 782 to 1316; 4096 x 4096 in 256 x 256 2510 to 2750 us; 16 of 1000 x 520 455, where 256 x 256 for the
// update alone would take 416.)
int form_of(const DeviceInfo &dev, int64_t count, int64_t m, int64_t n, bool symmetric, int64_t slices, int64_t other)
{
    // GEMM_GB300_ORTHOGONAL_FORM=0 to 3 (tests and sweeps): always this one; two digits: symmetric ones', the update's
    if (const char *e = std::getenv("GEMM_GB300_ORTHOGONAL_FORM"); e && *e >= '0' && *e <= '3') {
        const char c = !symmetric && e[1] >= '0' && e[1] <= '3' ? e[1] : *e;
        return c - '0';
    }
    int best = 0;
    double least = 1e300;
    static constexpr double kMore[4] = {5.5, 8.0, 10.5, 1.0}, kSlice[4] = {385.0, 365.0, 565.0, 380.0};
    for (int form = 0; form < 4; ++form) {
        const int64_t tm = tile_m(form), tn = tile_n(form), i = (m + tm - 1) / tm, j = (n + tn - 1) / tn;
        const int64_t tiles = count * (symmetric ? tm / tn * i * (i + 1) / 2 : i * j), room = is_pair(form) ? dev.num_sms / 2 : dev.num_sms;
        const double each = double(slices) + kMore[form] + (symmetric ? double(other) + kMore[form] : 0.0);
        const double cost = double((tiles + room - 1) / room) * each * kSlice[form];
        if (cost < least) {
            least = cost;
            best = form;
        }
    }
    return best;
}

struct ProductMaps {
    CUtensorMap a, b, out, in, turned_a, turned_b;
};

template <int FORM, int WHAT, bool F32>
cudaError_t launch_form(const DeviceInfo &dev, const ProductMaps &maps, StepParams p, int64_t columns, cudaStream_t stream)
{
    using S = Shape<FORM>;
    auto *kernel = orthogonal_kernel<FORM, WHAT, F32>;
    int room;
    if (S::kPair) {
        static std::atomic<int> cache[64];
        room = resident_pairs(kernel, kThreads, S::kBytes, dev.device, cache);
        if (room <= 0) return cudaErrorInitializationError;
    } else {
        const cudaError_t e = allow_smem_once(kernel, S::kBytes);
        if (e != cudaSuccess) return e;
        room = dev.num_sms;
    }
    p.tiles_m = int((p.n + S::kM - 1) / S::kM);
    p.tiles_n = int((columns + S::kN - 1) / S::kN);
    const int64_t per = WHAT <= kSquare ? int64_t(S::kM / S::kN) * p.tiles_m * (p.tiles_m + 1) / 2 : int64_t(p.tiles_m) * p.tiles_n;
    if (per * p.count >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    p.per = int(per);
    const int64_t units = per * p.count, grid = (units < room ? units : room) * (S::kPair ? 2 : 1);
    return launch_chained(kernel, dim3(unsigned(grid)), kThreads, S::kBytes, S::kPair ? 2 : 1, stream, maps.a, maps.b, maps.out, maps.in,
                          maps.turned_a, maps.turned_b, p);
}
template <int WHAT, bool F32 = false>
cudaError_t launch_product(const DeviceInfo &dev, int form, const ProductMaps &maps, const StepParams &p, int64_t columns, cudaStream_t stream)
{
    if (form == 0) return launch_form<0, WHAT, F32>(dev, maps, p, columns, stream);
    if (form == 1) return launch_form<1, WHAT, F32>(dev, maps, p, columns, stream);
    if (form == 2) return launch_form<2, WHAT, F32>(dev, maps, p, columns, stream);
    return launch_form<3, WHAT, F32>(dev, maps, p, columns, stream);
}

}  // namespace

cudaError_t launch_orthogonal_steps(const DeviceInfo &dev, const OrthogonalArgs &a, const OrthogonalLayout &l, const OrthogonalStep *plan,
                                    int steps, cudaStream_t stream)
{
    unsigned int *status = device_status_word(dev.device);
    if (status == nullptr || dev.smem_optin < size_t(kMostBytes)) return cudaErrorInitializationError;
    char *w = static_cast<char *>(a.work);
    StepParams p{};
    p.n = l.n;
    p.k = l.k;
    p.ldn = l.ldn;
    p.count = int(l.count);
    p.d = reinterpret_cast<float *>(w + l.dd);
    p.f = reinterpret_cast<float *>(w + l.df);
    p.Y = a.Y;
    p.ldy = a.ldy;
    p.stridey = a.stridey;
    p.y_rows = a.rows;
    p.y_cols = a.cols;
    p.y_bf16 = a.y_type == GEMM_TYPE_BF16;
    p.status = status;
    test_hooks(p.timeout_ns, p.inject_stall);
    const int slices_k = int((l.k + 63) / 64), slices_n = int((l.n + 63) / 64);
    // the square's tiles are the Gram matrix's: what it reads beside them must be stored
    const int symmetric = form_of(dev, l.count, l.n, l.n, true, slices_k * kProducts, slices_n * kProducts);
    const int wide = form_of(dev, l.count, l.n, l.k, false, slices_n * kProducts, 0);
    const int shift = is_pair(symmetric) ? 8 : 7;

    // X's two sets, in turn, E and F
    const int64_t planes = 2 * l.count;
    ProductMaps gram[2], square, update[2];
    CUtensorMap y_out;
    std::memset(&y_out, 0, sizeof(y_out));
    std::memset(&square, 0, sizeof(square));
    bool ok = make_map16(&square.a, w + l.e, l.n, l.n, l.ldn, planes, 128) &&
              make_map16(&square.b, w + l.e, l.n, l.n, l.ldn, planes, rows_b(symmetric)) &&
              make_map_columns(&square.turned_a, w + l.e, l.n, l.ldn, planes, 2) &&
              make_map_columns(&square.turned_b, w + l.e, l.n, l.ldn, planes, rows_b(symmetric) / 64) &&
              make_store_map(&square.in, w + l.e, GEMM_TYPE_F16, l.n, l.ldn, l.ldn, planes, l.n * l.ldn, true) &&
              make_store_map(&square.out, w + l.f, GEMM_TYPE_F16, l.n, l.ldn, l.ldn, planes, l.n * l.ldn, true);
    std::memset(update, 0, sizeof(update));
    ok = ok && make_map16(&update[0].a, w + l.f, l.n, l.n, l.ldn, planes, 128) &&
         make_map_columns(&update[0].turned_a, w + l.f, l.n, l.ldn, planes, 2);
    update[1] = update[0];
    std::memset(gram, 0, sizeof(gram));
    for (int i = 0; ok && i < (steps > 1 ? 2 : 1); ++i) {
        ok = make_map16(&gram[i].a, w + l.x[i], l.n, l.k, l.ldk, planes, 128) &&
             make_map16(&gram[i].b, w + l.x[i], l.n, l.k, l.ldk, planes, rows_b(symmetric)) &&
             make_map_columns(&update[i].b, w + l.x[i], l.n, l.ldk, planes, rows_b(wide) / 64) &&
             make_store_map(&update[i].in, w + l.x[i], GEMM_TYPE_F16, l.n, l.ldk, l.ldk, planes, l.n * l.ldk, true);
        gram[i].out = square.in;
    }
    if (!ok) return cudaErrorInvalidValue;
    update[0].out = update[1].in;
    update[1].out = update[0].in;
    p.y_tma = make_store_map(&y_out, a.Y, a.y_type, a.rows, a.cols, a.ldy, l.count, a.stridey, true);

    for (int i = 0; i < steps; ++i) {
        const OrthogonalStep &s = plan[i];
        p.a = s.a;
        p.b = s.b;
        p.c = s.c;
        const float *unit = i == 0 ? reinterpret_cast<const float *>(w + l.unit) : nullptr;
        StepParams q = p;
        q.num_kb = slices_k;
        q.unit = unit;
        q.from_acc = 1.0f / (s.x_scale * s.x_scale);
        q.to = s.e_scale;
        cudaError_t e = launch_product<kGram>(dev, symmetric, gram[i & 1], q, l.n, stream);
        if (e != cudaSuccess) return e;

        q = p;
        q.num_kb = slices_n;
        q.from_e = 1.0f / s.e_scale;
        q.from_acc = q.from_e * q.from_e;
        q.to = s.f_scale;
        q.shift_a = q.shift_b = shift;
        e = launch_product<kSquare>(dev, symmetric, square, q, l.n, stream);
        if (e != cudaSuccess) return e;

        q = p;
        q.num_kb = slices_n;
        q.unit = unit;
        q.from_x = 1.0f / s.x_scale;
        q.from_acc = q.from_x / s.f_scale;
        q.shift_a = shift;
        ProductMaps &maps = update[i & 1];
        if (i + 1 < steps) {
            q.to = s.next_scale;
            e = launch_product<kUpdate>(dev, wide, maps, q, l.k, stream);
        } else {
            q.to = 1.0f;
            maps.out = y_out;
            const bool turned = a.rows > a.cols;
            if (a.y_type == GEMM_TYPE_F32)
                e = turned ? launch_product<kResultTurned, true>(dev, wide, maps, q, l.k, stream)
                           : launch_product<kResult, true>(dev, wide, maps, q, l.k, stream);
            else
                e = turned ? launch_product<kResultTurned>(dev, wide, maps, q, l.k, stream)
                           : launch_product<kResult>(dev, wide, maps, q, l.k, stream);
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace gemm
