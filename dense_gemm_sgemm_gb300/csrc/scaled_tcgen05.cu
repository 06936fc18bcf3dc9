// Products of 8-bit matrices with an fp32 scale for every 128 elements along K, on the tcgen05 tensor
// cores (semantics: include/gemm_gb300.h):
//
//     C[m][n] = sum over K blocks kb of sa(m, kb) * sb(n, kb) * sum over k in kb of A[m][k] * B[n][k]
//
// A K block is one slice of the ring: its four MMAs (kind::f8f6f4, K = 32) start a fresh accumulator in
// tensor memory, and eight warps read it back, scale it and add it to fp32 sums in their registers, while
// the MMAs of the next block fill another accumulator.  The tensor cores thus sum 128 products, whose terms
// are exact, and everything longer is summed in fp32 on the CUDA cores with any fp32 scales, not only powers
// of two.  A lane of tensor memory is one row of A, so its scale is one value a thread; B's are one a column
// (COLS), read from shared memory beside the sums, or one for all 128 columns, multiplied into the row's before.
//
// Two forms.  Pairs: two CTAs on neighbouring SMs, 256 x 256 tiles (cta_group::2), persistent, C stored by
// TMA; the eight adding warps share a block's columns.  Tiles: one CTA a tile of 128 x BN, K split over a cluster
// of up to eight CTAs whose sums meet in distributed shared memory; the adding warps form two groups that take
// blocks in turn.  Tiles take problems without enough tiles for the pairs, and the tiles beyond the pairs' last
// full wave.  With few rows of A (or B) the host swaps the operands: the long side takes the 128 lanes, the short
// one the BN columns.
//
// What bounds them (GB300).  Pairs, 16384 x 4096 x 4096, B's scales by 128 x 128: 209 to 221 us (the device's temperature), 2490
// to 2630 TFLOP/s, about 900 SM cycles a block, of which the MMAs need 512 and the copies from L2 (64 KB a pair) 625: the adding warps, which
// read 256 columns of all lanes from tensor memory and issue as many multiply-adds; with a scale for every column
// of B 319 us, since each pair of sums takes a product more and its scales from shared memory.  4096 x 4096 x 8192,
// scales of both by column, fp32 out: 183 us in pairs alone, 168 with the last wave's 28 tiles in single CTAs.
// Tiles: latency: 1 x 4096 x 4096 6.9 us (2.4 TB/s of weight), 64 x 8192 x 4096 10.6 (3.2 TB/s), 512 x 4096 x 1024
// 8.2: 4 to 5 us of launch, first copies, and joining and storing the sums, and 0.2 to 0.35 us a block.
// Tried and dropped: 16 adding warps of 64 columns each (242 us, registers too few), 256-column pieces, loads of the
// scales to registers (750 cycles a block whatever its size), one-lane producers and issuers in the pair kernel
// (the adding warps then spill more).
//
// Every wait is bounded: when one expires the kernel raises the device's error word, stops all roles, waits
// (bounded) for its own copies and MMAs in flight, frees its TMEM and returns.
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "scaled_internal.h"
#include "tcgen05_ptx.cuh"
#include "tcgen05_roles.cuh"
#include "tensor_map.h"

namespace gemm {
namespace {

constexpr int kEpiWarps = 8;  // adding warps
// The pair kernel's warps come in fours, so that the adding ones may have more registers than the launch
// gives each: (4 * 72 + 8 * 216) * 32 = 12 * 32 * 168.
constexpr int kPairFirst = 4, kPairThreads = 32 * (kPairFirst + kEpiWarps);
constexpr int kBox = 128 * 128;  // bytes: 128 rows of a K block, or its 128 k of 128 rows
constexpr unsigned kFull = 0xffffffffu;

struct ScaledParams {
    int64_t M, N;
    int num_kb, tiles_m, tiles_n, splits;
    int tiles;               // of a pair's, that pairs take
    int tail;                // the first of them that single CTAs take, or -1: their tiles are a grid of their own
    int a_mn, b_mn;          // operands stored K x M, K x N
    uint32_t formats;        // their 8-bit types in the instruction descriptor
    const float *sa, *sb;
    int64_t sa_mn, sa_k, sb_mn, sb_k;
    int a_shift, b_shift;    // 7: a scale for 128 rows
    void *C;
    int64_t ldc;
    int c_type, transposed;  // transposed: C is N x M
    int c_tma;
    unsigned int *status;
    uint64_t timeout_ns;
    int inject_stall;  // test hook: the producer never fills its first slice
};

// ------------------------------------------------------------------ PTX
template <bool PAIR>
__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (PAIR)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                     : "memory");
}

// 16 or 32 columns of this thread's TMEM lane, on their way: not to be read before tmem_arrived().
__device__ __forceinline__ void tmem_start(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_start(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
                   "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
                   "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}
// Waits for the loads started so far; the registers pass through it, so that nothing reads them earlier.
__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

// ------------------------------------------------------------------ scaling and adding a K block
// Scales whose products with each other and with a block's sum (2^-32 to 2^39) stay well inside fp32.
__device__ __forceinline__ bool mild(float s)
{
    const float a = fabsf(s);
    return a == 0.0f || (a >= 0x1p-40f && a <= 0x1p40f);
}
// s as two factors of half its exponent each (zero, infinite and NaN scales as 1 and s), the second one below 2^64,
// so that the product of two of them is finite.  A block's sum times both scales' first factors and then both second
// ones stays in fp32's range wherever the result does.  (Two first factors of 2^64, rounded towards zero, are fp32's
// largest value, so that a sum of zero stays zero; any other is beyond fp32's range either way.)
__device__ __forceinline__ float2 halves(float s)
{
    const float a = fabsf(s);
    if (!(a > 0.0f && a <= FLT_MAX)) return make_float2(1.0f, s);
    const int e = (ilogbf(s) + 1) >> 1;
    return make_float2(__uint_as_float(uint32_t(127 + e) << 23), s * __uint_as_float(uint32_t(127 - e) << 23));
}

__device__ __forceinline__ float2 pair_of(uint32_t x, uint32_t y) { return make_float2(__uint_as_float(x), __uint_as_float(y)); }
__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }

// ------------------------------------------------------------------ scales
// A K block's scales pass through shared memory, in slots of their own: one warp or two copy them (cp.async,
// any strides), look at a block's when those of a few blocks behind it are on their way, and announce it.
// (With loads to the adding warps' registers one or two blocks ahead a block took 750 SM cycles whatever its
// size; with those warps looking at them 400 more than now; one warp for a pair's scales took 850 a block.)
// The adding warps release a block's slot when they have read the next block.  The ring's barriers would not
// do: the MMAs do not wait for scales, so a stage's barrier could complete twice before this warp looks.
// Whether two phases are complete, and a wait for both: all lanes with one answer.
__device__ __forceinline__ bool both_there(uint32_t bar0, uint32_t phase0, uint32_t bar1, uint32_t phase1)
{
    const bool there = mbar_try_wait(bar0, phase0) & mbar_try_wait(bar1, phase1);
    return __all_sync(kFull, there) != 0;
}
__device__ __forceinline__ bool wait_both(const Watch &watch, uint32_t bar0, uint32_t phase0, uint32_t bar1, uint32_t phase1)
{
    const bool got = watch.wait(bar0, phase0) && watch.wait(bar1, phase1);
    return __all_sync(kFull, got) != 0;
}

// Floats of a slot: row scales, column scales (without COLS those of the two runs of 128 columns), and what the
// adding warps multiply a row by: its scale, or without COLS its products with the column scales (PAIRS: with
// either run's); NaN in all rows where some scale is not mild, which sends the warps to the scales themselves.
template <bool COLS, bool PAIRS> struct Slot {
    static constexpr int kEach = !COLS && PAIRS ? 2 : 1, kCols = 128, kRow = kCols + (COLS ? (PAIRS ? 256 : 128) : 4);
    static constexpr int kFloats = kRow + 128 * kEach;
};

__device__ __forceinline__ void copy_scale(float *dst, const float *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ int64_t scale_row(int64_t row, int64_t rows) { return row < rows ? row : rows - 1; }

// A warp that handles a tile's scales: one block in STEP.  BN: columns of the tile;  DELAY: of its blocks that
// are on their way while it looks at one.
template <bool COLS, bool PAIRS, int BN, int SLOTS, int STEP, int DELAY> struct ScaleCopies {
    using L = Slot<COLS, PAIRS>;
    static constexpr int kColumns = COLS ? BN / 32 : 1;
    static_assert(SLOTS % STEP == 0, "every warp has slots of its own");
    float *slots;
    uint32_t full0, empty0;  // barriers of the slots, one arrival each and the adding warps'
    int lane, copying, looking, behind = 0;
    uint32_t phase = 1;  // of the slots' release
    const float *rows[4], *columns[kColumns];  // of the next block
    int64_t step_a, step_b;

    __device__ __forceinline__ ScaleCopies(float *s, uint32_t full, uint32_t empty, int l, int first)
        : slots(s), full0(full), empty0(empty), lane(l), copying(first), looking(first)
    {
    }
    // The tile's rows of scales (rows outside the matrix take the last one's), from block kb.
    __device__ __forceinline__ void begin(const ScaledParams &p, int64_t m0, int64_t n0, int kb)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) rows[i] = p.sa + (scale_row(m0 + i * 32 + lane, p.M) >> p.a_shift) * p.sa_mn + kb * p.sa_k;
#pragma unroll
        for (int i = 0; i < kColumns; ++i) {
            // PAIRS: a piece's columns side by side: 64 from column 64 h of the tile, 64 from column 128 + 64 h
            const int at = !COLS ? (PAIRS ? 128 * (lane & 1) : 0) : PAIRS ? (i & 1) * 32 + (i >> 1 & 1) * 128 + (i >> 2) * 64 : i * 32;
            columns[i] = p.sb + (scale_row(n0 + at + (COLS ? lane : 0), p.N) >> p.b_shift) * p.sb_mn + kb * p.sb_k;
        }
        step_a = STEP * p.sa_k;
        step_b = STEP * p.sb_k;
    }
    __device__ __forceinline__ bool copy(const Watch &watch)
    {
        if (!__all_sync(kFull, watch.wait(empty0 + 8u * copying, phase))) return false;
        float *slot = slots + copying * L::kFloats;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            copy_scale(slot + i * 32 + lane, rows[i]);
            rows[i] += step_a;
        }
#pragma unroll
        for (int i = 0; i < kColumns; ++i) {
            if (COLS || lane < 2) copy_scale(slot + L::kCols + i * 32 + lane, columns[i]);
            columns[i] += step_b;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        copying += STEP;
        if (copying >= SLOTS) {
            copying -= SLOTS;
            phase ^= 1u;
        }
        if (++behind > DELAY) {
            asm volatile("cp.async.wait_group %0;" ::"n"(DELAY) : "memory");
            look();
        }
        return true;
    }
    __device__ __forceinline__ void finish()
    {
        asm volatile("cp.async.wait_all;" ::: "memory");
        while (behind > 0) look();
    }
    __device__ __forceinline__ void look()
    {
        float *slot = slots + looking * L::kFloats;
        __syncwarp();
        bool fine = true;
        float row[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            row[i] = slot[i * 32 + lane];
            fine = fine && mild(row[i]);
        }
        float c0 = 1.0f, c1 = 1.0f;
        if (COLS) {
#pragma unroll
            for (int i = 0; i < BN; i += 32) fine = fine && mild(slot[L::kCols + i + lane]);
        } else {
            c0 = slot[L::kCols];
            c1 = slot[L::kCols + 1];
            fine = fine && mild(c0) && mild(c1);
        }
        if (!__all_sync(kFull, fine)) c0 = c1 = __uint_as_float(0x7fffffffu);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float *to = slot + L::kRow + L::kEach * (i * 32 + lane);
            if (L::kEach == 2) *reinterpret_cast<float2 *>(to) = make_float2(row[i] * c0, row[i] * c1);
            else *to = row[i] * c0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(full0 + 8u * looking);
        looking = looking + STEP >= SLOTS ? looking + STEP - SLOTS : looking + STEP;
        --behind;
    }
};

// The sums of one thread: a row of A, CW columns of B.  sb is the block's column scales (COLS), or one for
// each run of 64 columns (PAIRS) or for all.
template <int CW, bool COLS, bool PAIRS> struct Sums {
    static constexpr int kChunk = PAIRS && !COLS ? 32 : 16, kChunks = CW / kChunk;
    float2 at[CW / 2];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < CW / 2; ++i) at[i] = make_float2(0.0f, 0.0f);
    }
    // Adds columns c .. : v * s * (the columns' scales, COLS).
    __device__ __forceinline__ void add_chunk(int c, const uint32_t (&v)[kChunk], float s, const float *sb)
    {
        if constexpr (COLS) {
#pragma unroll
            for (int i = 0; i < kChunk; i += 4) {
                const float4 w = *reinterpret_cast<const float4 *>(sb + c + i);
                float2 &lo = at[(c + i) / 2], &hi = at[(c + i) / 2 + 1];
                lo = __ffma2_rn(pair_of(v[i], v[i + 1]), __fmul2_rn(make_float2(w.x, w.y), twice(s)), lo);
                hi = __ffma2_rn(pair_of(v[i + 2], v[i + 3]), __fmul2_rn(make_float2(w.z, w.w), twice(s)), hi);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kChunk; i += 2) at[(c + i) / 2] = __ffma2_rn(pair_of(v[i], v[i + 1]), twice(s), at[(c + i) / 2]);
        }
    }
    // Adds the block in the accumulator at taddr.  row: of the tile's 128;  part: the first of the warp's
    // columns;  scratch: 2 * CW floats of the warp's own.  `peek` is called while its last columns are on their
    // way (the answer to whether the next block is there takes as long), `read` once it has been read.
    template <class Peek, class Read>
    __device__ __forceinline__ void add(uint32_t taddr, const float *slot, int row, int part, float *scratch, int lane, Peek peek, Read read)
    {
        using L = Slot<COLS, PAIRS>;
        uint32_t r[2][kChunk];
        tmem_start(taddr, r[0]);
        const float *sb = slot + L::kCols + (COLS ? part : 0);
        float s0, s1;
        if (L::kEach == 2) {
            const float2 t = *reinterpret_cast<const float2 *>(slot + L::kRow + 2 * row);
            s0 = t.x;
            s1 = t.y;
        } else {
            s0 = s1 = slot[L::kRow + row];
        }
        if (__builtin_expect(s0 != s0, 0)) {
            add_any(taddr, slot[row], sb, scratch, lane);
            read();
            peek();
            return;
        }
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            tmem_arrived(r[i & 1]);
            if (i + 1 < kChunks) tmem_start(taddr + (i + 1) * kChunk, r[(i + 1) & 1]);
            else read();
            if (i + 2 == kChunks || kChunks == 1) peek();
            add_chunk(i * kChunk, r[i & 1], PAIRS && i * kChunk >= 64 ? s1 : s0, sb);
        }
    }
    // The same for scales of any size: first factors, then second ones.
    __device__ __forceinline__ void add_any(uint32_t taddr, float s, const float *sb, float *scratch, int lane)
    {
        constexpr int kScales = COLS ? CW : 2;
        const float2 h = halves(s);
        __syncwarp();  // the block before it has been added
        for (int i = lane; i < kScales; i += 32) {
            const float2 f = halves(sb[i]);
            scratch[i] = f.y;
            scratch[CW + i] = f.x;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            uint32_t v[kChunk];
            tmem_start(taddr + i * kChunk, v);
            tmem_arrived(v);
            const int run = PAIRS ? i * kChunk / 64 : 0;
#pragma unroll
            for (int j = 0; j < kChunk; ++j)
                v[j] = __float_as_uint(__uint_as_float(v[j]) * __fmul_rz(h.x, scratch[CW + (COLS ? i * kChunk + j : run)]));
            add_chunk(i * kChunk, v, COLS ? h.y : h.y * scratch[run], scratch);
        }
    }
};

// ------------------------------------------------------------------ copies
// The box of an operand for block kb: 128 rows from mn0 (rows of the tensor map), or, stored K x MN, the
// block's 128 rows from column mn0.
template <bool PAIR>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, uint32_t bar, int mn, int mn0, int kb)
{
    const int c0 = mn ? mn0 : kb * 128, c1 = mn ? kb * 128 : mn0;
    if (PAIR) tma_load_3d_pair(dst, map, bar, c0, c1, 0);
    else tma_load_3d(dst, map, bar, c0, c1, 0);
}
// Descriptor of such a box (stored K x MN its 128 columns are one 128-byte atom wide: no leading offset), and
// its step from one K = 32 to the next.
__device__ __forceinline__ uint64_t box_desc(uint32_t addr) { return smem_desc(addr, 16, 1024); }
__device__ __forceinline__ uint32_t box_step(int mn) { return (mn ? 32 * 128 : 32) >> 4; }

__device__ __forceinline__ uint32_t f8_idesc(const ScaledParams &p, int n, int m) { return make_idesc(p.a_mn, p.b_mn, n, m) | p.formats; }

// ------------------------------------------------------------------ pairs
// 256 x 256 tiles.  A K block's product is formed in two pieces of 128 columns (64 of either CTA's half of B),
// each in one of two accumulators, so that while the four warps of one piece read theirs the tensor cores are
// at the other.  Piece h's column j is column (j / 64) * 128 + 64 h + j % 64 of the tile.
//
// The second piece's commit, on the stage's `empty` barrier, tells the producer that the boxes may be
// overwritten as well as the adding warps that the accumulator is full.  (A warp that waits for one phase of
// it cannot miss it: the stage is used again only after the warp has released an accumulator that comes later.)
template <bool COLS> struct PairSmem {
    static constexpr int kStages = 5, kStage = 2 * kBox;
    static constexpr int kSlot = Slot<COLS, true>::kFloats, kSlots = 8;
    static constexpr int kEpi = kEpiWarps * 4096, kScratch = kEpiWarps * 2 * 128 * 4, kBars = 512;
    static constexpr int kBytes = kStages * kStage + kEpi + kScratch + kSlots * kSlot * 4 + kBars + 1024;
    static_assert(kBytes <= 227 * 1024, "one CTA per SM");
    uint32_t ring, bar0;
    uint8_t *epi;
    float *scratch, *scales;
    volatile uint32_t *tmem_slot;
    volatile int *abort_flag;
    __device__ __forceinline__ explicit PairSmem(uint8_t *raw)
    {
        const uint32_t r = smem_u32(raw), base = (r + 1023u) & ~1023u;
        uint8_t *p = raw + (base - r);
        ring = base;
        epi = p + kStages * kStage;
        uint8_t *bars = epi + kEpi;
        bar0 = smem_u32(bars);
        tmem_slot = reinterpret_cast<volatile uint32_t *>(bars + kBars - 16);
        abort_flag = reinterpret_cast<volatile int *>(bars + kBars - 8);
        scales = reinterpret_cast<float *>(bars + kBars);
        scratch = scales + kSlots * kSlot;
    }
    __device__ __forceinline__ uint32_t full(int s) const { return bar0 + 8u * s; }
    __device__ __forceinline__ uint32_t empty(int s) const { return bar0 + 8u * (kStages + s); }
    __device__ __forceinline__ uint32_t acc_empty(int i) const { return bar0 + 8u * (2 * kStages + i); }
    __device__ __forceinline__ uint32_t first_full(int i) const { return bar0 + 8u * (2 * kStages + 4 + i); }
    __device__ __forceinline__ uint32_t scale_full(int i) const { return bar0 + 8u * (2 * kStages + 6 + i); }
    __device__ __forceinline__ uint32_t scale_empty(int i) const { return bar0 + 8u * (2 * kStages + 6 + kSlots + i); }
    __device__ __forceinline__ uint32_t drain() const { return bar0 + 8u * (2 * kStages + 6 + 2 * kSlots); }
    __device__ __forceinline__ uint32_t a(int s) const { return ring + uint32_t(s * kStage); }
    __device__ __forceinline__ uint32_t b(int s) const { return a(s) + kBox; }
};

// Tile t of the visiting order, groups of eight tile rows column by column (raster() in 32 bits).
__device__ __forceinline__ void tile_of(unsigned t, unsigned tiles_m, unsigned tiles_n, int &tm, int &tn)
{
    const unsigned group = t / (8 * tiles_n), r = t - group * 8 * tiles_n, rows = min(8u, tiles_m - 8 * group);
    tm = int(8 * group + r % rows);
    tn = int(r / rows);
}

template <bool COLS, bool F32>
__global__ void __launch_bounds__(kPairThreads, 1)
scaled_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_c, const __grid_constant__ ScaledParams p)
{
    extern __shared__ uint8_t smem_raw[];
    using Smem = PairSmem<COLS>;
    const Smem sh(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < Smem::kStages; ++s) {
            mbar_init(sh.full(s), 1);
            mbar_init(sh.empty(s), 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(sh.acc_empty(i), kEpiWarps);  // a piece's four warps of both CTAs
        for (int i = 0; i < 2; ++i) mbar_init(sh.first_full(i), 1);
        for (int i = 0; i < Smem::kSlots; ++i) {
            mbar_init(sh.scale_full(i), 1);
            mbar_init(sh.scale_empty(i), kEpiWarps);
        }
        mbar_init(sh.drain(), 1);
        *sh.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    cluster_sync();
    if (warp == 1) tmem_alloc<true>(smem_u32(const_cast<uint32_t *>(sh.tmem_slot)), 512);
    chain_wait();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *sh.tmem_slot;
    const Watch watch{sh.abort_flag, p.status, p.timeout_ns};
    const int tiles = p.tiles, first = int(cluster_id_x()), step = int(cluster_count_x());
    Ring ring(Smem::kStages);
    bool ok = true;

    if (warp < kPairFirst) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;" ::: "memory");
        if (warp == 0) {
            // ---------------- producer: this CTA's 128 rows of A and its 128 of the tile's 256 rows of B
            const bool leader = elect_one();
            const uint32_t full0 = map_to_rank(sh.full(0), 0);
            if (leader) {
                tma_prefetch_desc(&map_a);
                tma_prefetch_desc(&map_b);
            }
            for (int t = first; ok && t < tiles; t += step) {
                int tm, tn;
                tile_of(t, p.tiles_m, p.tiles_n, tm, tn);
                const int m0 = tm * 256 + int(rank) * 128, n0 = tn * 256;
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    ok = watch.wait(sh.empty(ring.stage), ring.phase ^ 1u);
                    if (__any_sync(kFull, !ok)) {
                        ok = false;
                        break;
                    }
                    if (leader) {
                        if (rank == 0) mbar_expect_tx(sh.full(ring.stage), 2 * Smem::kStage);
                        if (!(p.inject_stall && kb == 0 && t == first)) {
                            const uint32_t full = full0 + 8u * ring.stage;
                            load_box<true>(sh.a(ring.stage), &map_a, full, p.a_mn, m0, kb);
                            load_box<true>(sh.b(ring.stage), &map_b, full, p.b_mn, n0 + int(rank) * 128, kb);
                        }
                    }
                    __syncwarp();
                    ring.next();
                }
            }
            if (leader) {
                if (!ok) {  // copies in flight get time to land
                    const uint64_t t0 = global_timer_ns();
                    while (global_timer_ns() - t0 < 2000000ull) {
                    }
                } else {  // no commit is on its way to this CTA's barriers when it exits
                    for (int i = 0; i < Smem::kStages; ++i) {
                        if (!watch.wait(sh.empty(ring.stage), ring.phase ^ 1u)) break;
                        ring.next();
                    }
                }
            }
        } else if (warp >= 2) {
            // ---------------- scales of this CTA's rows of A and of all the tile's of B: two warps, in turn
            const int mine = warp - 2;
            ScaleCopies<COLS, true, 256, Smem::kSlots, 2, 1> copies(sh.scales, sh.scale_full(0), sh.scale_empty(0), lane, mine);
            int turn = 0;
            for (int t = first; ok && t < tiles; t += step) {
                int tm, tn;
                tile_of(t, p.tiles_m, p.tiles_n, tm, tn);
                copies.begin(p, int64_t(tm) * 256 + rank * 128, int64_t(tn) * 256, turn ^ mine);
                for (int kb = 0; ok && kb < p.num_kb; ++kb, turn ^= 1)
                    if (turn == mine) ok = copies.copy(watch);
            }
            copies.finish();
        } else if (warp == 1 && rank == 0) {
            // ---------------- MMA issuer
            const bool leader = elect_one();
            const uint32_t idesc = f8_idesc(p, 128, 256), step_a = box_step(p.a_mn), step_b = box_step(p.b_mn);
            const uint64_t a0 = box_desc(sh.a(0)), b0 = box_desc(sh.b(0));
            const uint32_t piece_b = (p.b_mn ? 64 : 64 * 128) >> 4;  // 64 columns of a box, or 64 rows
            int acc = 0;
            uint32_t acc_phase = 0;
            for (int t = first; ok && t < tiles; t += step)
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    ok = watch.wait(sh.full(ring.stage), ring.phase);
                    if (!ok) break;
                    const uint64_t a = a0 + uint32_t(ring.stage * (Smem::kStage >> 4));
                    const uint64_t b = b0 + uint32_t(ring.stage * (Smem::kStage >> 4));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        ok = ok && watch.wait<true>(sh.acc_empty(2 * acc + h), acc_phase ^ 1u);
                        if (!ok) break;
                        tc_fence_after();
                        if (leader) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                umma_f8<true>(tmem + uint32_t((2 * acc + h) * 128), a + k * step_a, b + h * piece_b + k * step_b, idesc,
                                              k > 0 ? 1u : 0u);
                            commit_both(h == 0 ? sh.first_full(acc) : sh.empty(ring.stage));
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    ring.next();
                    acc ^= 1;
                    acc_phase ^= acc == 0 ? 1u : 0u;
                }
            if (!ok && leader) {  // MMAs in flight finish before TMEM is released
                umma_commit<true>(sh.drain());
                const volatile int no_abort = 0;
                mbar_wait(sh.drain(), 0, &no_abort, 100000000ull);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;" ::: "memory");
        // ---------------- adding warps: rows 32 * quarter .. of this CTA's 128, one piece's columns
        const int quarter = warp & 3, half = (warp - kPairFirst) >> 2;
        Staging<F32> staging(sh.epi + (warp - kPairFirst) * 4096, lane);
        float *scratch = sh.scratch + (warp - kPairFirst) * 2 * 128;
        const uint32_t acc_empty0 = map_to_rank(sh.acc_empty(half), 0);
        const uint32_t taddr0 = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(half * 128);
        Ring slot(Smem::kSlots);
        int acc = 0, added = -1;  // added: the slot of the block before
        uint32_t acc_phase = 0;
        for (int t = first; ok && t < tiles; t += step) {
            int tm, tn;
            tile_of(t, p.tiles_m, p.tiles_n, tm, tn);
            const int64_t m0 = int64_t(tm) * 256 + rank * 128 + quarter * 32, n0 = int64_t(tn) * 256 + half * 64;
            Sums<128, COLS, true> sums;
            sums.clear();
            bool there = false;
            for (int kb = 0; kb < p.num_kb; ++kb) {
                // of the next block: its slot, and the barrier and phase of its accumulator
                auto scales = [&] { return sh.scale_full(slot.stage); };
                auto full = [&] { return half == 0 ? sh.first_full(acc) : sh.empty(ring.stage); };
                auto phase = [&] { return half == 0 ? acc_phase : ring.phase; };
                if (!there) ok = wait_both(watch, scales(), slot.phase, full(), phase());
                if (!ok) break;
                tc_fence_after();
                const float *at = sh.scales + slot.stage * Smem::kSlot;
                const int now = acc, reading = slot.stage;
                ring.next();
                slot.next();
                acc ^= 1;
                acc_phase ^= acc == 0 ? 1u : 0u;
                sums.add(
                    taddr0 + uint32_t(now * 256), at, quarter * 32 + lane, half * 128, scratch, lane,
                    [&] { there = kb + 1 < p.num_kb && both_there(scales(), slot.phase, full(), phase()); },
                    [&] {
                        release_accumulator(acc_empty0 + 16u * now, lane);
                        if (lane == 0 && added >= 0) mbar_arrive(sh.scale_empty(added));
                        added = reading;
                    });
            }
            if (!ok) break;
            if (m0 >= p.M) continue;
#pragma unroll
            for (int c = 0; c < 128; c += 32) {
                const int64_t n = n0 + (c / 64) * 128 + c % 64;
                if (n >= p.N) break;
                float v[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    v[2 * i] = sums.at[c / 2 + i].x;
                    v[2 * i + 1] = sums.at[c / 2 + i].y;
                }
                store_rows(staging, v, &map_c, p.c_tma != 0, p.C, p.ldc, m0, n, p.M, p.N, p.c_type == GEMM_TYPE_BF16, 0);
            }
        }
        staging.finish();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves or frees TMEM while the other may still use it
    tc_fence_after();
    if (warp == 1) tmem_free<true>(tmem, 512);
}

// ------------------------------------------------------------------ tiles
// One CTA: 128 rows of A, BN of B, the K blocks of its rank in the cluster.
template <int BN> struct TileSmem {
    static constexpr int kFirst = 4, kThreads = 32 * (kFirst + kEpiWarps);
    static constexpr int kStage = kBox + BN * 128, kStages = BN == 128 ? 6 : BN == 64 ? 8 : 9;
    static constexpr int kBuffers = 4, kTmem = BN * kBuffers;
    static constexpr int kRow = BN + 4;  // floats of a row of sums: 16-byte stores by rows without bank conflicts
    static constexpr int kSlot = Slot<true, false>::kFloats > Slot<false, false>::kFloats ? Slot<true, false>::kFloats : Slot<false, false>::kFloats;
    static constexpr int kSlots = 8;
    static constexpr int kBars = 512, kScratch = kEpiWarps * 2 * BN * 4;
    static constexpr int kBytes = kStages * kStage + kScratch + kSlots * kSlot * 4 + kBars + 1024;
    static_assert(128 * kRow * 4 <= kStages * kStage && kBytes <= 227 * 1024, "one CTA per SM");
    uint32_t ring, bar0;
    float *scratch, *scales;
    float *sums;  // in the ring's place, once it is empty
    volatile uint32_t *tmem_slot;
    volatile int *abort_flag;
    __device__ __forceinline__ explicit TileSmem(uint8_t *raw)
    {
        const uint32_t r = smem_u32(raw), base = (r + 1023u) & ~1023u;
        uint8_t *p = raw + (base - r);
        ring = base;
        sums = reinterpret_cast<float *>(p);
        uint8_t *bars = p + kStages * kStage;
        bar0 = smem_u32(bars);
        tmem_slot = reinterpret_cast<volatile uint32_t *>(bars + kBars - 16);
        abort_flag = reinterpret_cast<volatile int *>(bars + kBars - 8);
        scales = reinterpret_cast<float *>(bars + kBars);
        scratch = scales + kSlots * kSlot;
    }
    __device__ __forceinline__ uint32_t full(int s) const { return bar0 + 8u * s; }
    __device__ __forceinline__ uint32_t empty(int s) const { return bar0 + 8u * (kStages + s); }
    __device__ __forceinline__ uint32_t acc_empty(int i) const { return bar0 + 8u * (2 * kStages + i); }
    __device__ __forceinline__ uint32_t scale_full(int i) const { return bar0 + 8u * (2 * kStages + kBuffers + i); }
    __device__ __forceinline__ uint32_t scale_empty(int i) const { return bar0 + 8u * (2 * kStages + kBuffers + kSlots + i); }
    __device__ __forceinline__ uint32_t drain() const { return bar0 + 8u * (2 * kStages + kBuffers + 2 * kSlots); }
    __device__ __forceinline__ uint32_t a(int s) const { return ring + uint32_t(s * kStage); }
    __device__ __forceinline__ uint32_t b(int s) const { return a(s) + kBox; }
};

template <class T>
__device__ __forceinline__ void store4(T *to, const float4 v, int64_t left)
{
    const float e[4] = {v.x, v.y, v.z, v.w};
    if (left >= 4) {
        T out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = from_f32<T>(e[i]);
        if constexpr (sizeof(T) == 4) *reinterpret_cast<float4 *>(to) = v;
        else *reinterpret_cast<uint2 *>(to) = *reinterpret_cast<const uint2 *>(out);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) to[i] = from_f32<T>(e[i]);
    }
}

// C from the sums of the cluster's CTAs, added in the order of K: this CTA's share of the tile's 128 rows.
template <class T, int BN>
__device__ __forceinline__ void store_tile(const ScaledParams &p, const float *sums, uint32_t rank, int64_t m0, int64_t n0)
{
    constexpr int kRow = BN + 4;
    const int height = 128 / p.splits, top = int(rank) * height;
    uint32_t base[8];
#pragma unroll
    for (int s = 0; s < 8; ++s) base[s] = s < p.splits ? map_to_rank(smem_u32(sums), uint32_t(s)) : 0u;
    T *C = static_cast<T *>(p.C);
    for (int i = threadIdx.x; i < height * BN / 4; i += TileSmem<BN>::kThreads) {
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        int row, col;  // of the piece: four columns of a row, or transposed four rows of a column
        if (p.transposed) {
            row = top + i % (height / 4) * 4;
            col = i / (height / 4);
        } else {
            row = top + i / (BN / 4);
            col = i % (BN / 4) * 4;
        }
        if (m0 + row >= p.M || n0 + col >= p.N) continue;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            if (s >= p.splits) break;
            if (p.transposed) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float f;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(base[s] + uint32_t((row + j) * kRow + col) * 4u) : "memory");
                    v[j] += f;
                }
            } else {
                float4 f;
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
                             : "r"(base[s] + uint32_t(row * kRow + col) * 4u)
                             : "memory");
                v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
            }
        }
        const float4 out = make_float4(v[0], v[1], v[2], v[3]);
        if (p.transposed) store4<T>(C + (n0 + col) * p.ldc + m0 + row, out, p.M - m0 - row);
        else store4<T>(C + (m0 + row) * p.ldc + n0 + col, out, p.N - n0 - col);
    }
}

template <int BN, bool COLS>
__global__ void __launch_bounds__(TileSmem<BN>::kThreads, 1)
scaled_tile_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ ScaledParams p)
{
    extern __shared__ uint8_t smem_raw[];
    using Smem = TileSmem<BN>;
    const Smem sh(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = p.splits > 1 ? cluster_ctarank() : 0u;
    const int tile = int(blockIdx.x) / p.splits;
    int64_t m0, n0;
    if (p.tail < 0) {
        m0 = int64_t(tile % p.tiles_m) * 128;
        n0 = int64_t(tile / p.tiles_m) * BN;
    } else {  // a quarter of a pair's tile
        int tm, tn;
        tile_of(p.tail + tile / 4, p.tiles_m, p.tiles_n, tm, tn);
        m0 = int64_t(tm) * 256 + (tile & 1) * 128;
        n0 = int64_t(tn) * 256 + (tile & 2) * 64;
        if (m0 >= p.M || n0 >= p.N) return;  // with its whole cluster
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < Smem::kStages; ++s) {
            mbar_init(sh.full(s), 1);
            mbar_init(sh.empty(s), 1);
        }
        for (int i = 0; i < Smem::kBuffers; ++i) mbar_init(sh.acc_empty(i), kEpiWarps / 2);
        for (int i = 0; i < Smem::kSlots; ++i) {
            mbar_init(sh.scale_full(i), 1);
            mbar_init(sh.scale_empty(i), kEpiWarps / 2);
        }
        mbar_init(sh.drain(), 1);
        *sh.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<false>(smem_u32(const_cast<uint32_t *>(sh.tmem_slot)), Smem::kTmem);
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&map_a);
        tma_prefetch_desc(&map_b);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (p.tail < 0) {
        chain_wait();
    } else {  // after pairs: nothing is read that they write, and they let this kernel begin when all ahead of them had ended
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        __threadfence();
    }
    const uint32_t tmem = *sh.tmem_slot;
    const Watch watch{sh.abort_flag, p.status, p.timeout_ns};
    const int kb0 = int(int64_t(p.num_kb) * rank / p.splits), kb1 = int(int64_t(p.num_kb) * (rank + 1) / p.splits);
    Ring ring(Smem::kStages);
    bool ok = true;

    if (warp < Smem::kFirst) {
        if (BN == 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;" ::: "memory");
        if (warp == 0) {
            // ---------------- producer, one lane
            if (elect_one()) {
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = watch.wait(sh.empty(ring.stage), ring.phase ^ 1u);
                    if (!ok) break;
                    mbar_expect_tx(sh.full(ring.stage), Smem::kStage);
                    if (!(p.inject_stall && kb == kb0)) {
                        load_box<false>(sh.a(ring.stage), &map_a, sh.full(ring.stage), p.a_mn, int(m0), kb);
                        load_box<false>(sh.b(ring.stage), &map_b, sh.full(ring.stage), p.b_mn, int(n0), kb);
                    }
                    ring.next();
                }
                if (!ok) {  // copies in flight get time to land
                    const uint64_t t0 = global_timer_ns();
                    while (global_timer_ns() - t0 < 2000000ull) {
                    }
                }
            }
        } else if (warp == 1) {
            // ---------------- MMA issuer, one lane
            if (elect_one()) {
                const uint32_t idesc = f8_idesc(p, BN, 128), step_a = box_step(p.a_mn), step_b = box_step(p.b_mn);
                const uint64_t a0 = box_desc(sh.a(0)), b0 = box_desc(sh.b(0));
                Ring acc(Smem::kBuffers);
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = watch.wait(sh.acc_empty(acc.stage), acc.phase ^ 1u);
                    ok = ok && watch.wait(sh.full(ring.stage), ring.phase);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t a = a0 + uint32_t(ring.stage * (Smem::kStage >> 4));
                    const uint64_t b = b0 + uint32_t(ring.stage * (Smem::kStage >> 4));
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_f8<false>(tmem + uint32_t(acc.stage * BN), a + k * step_a, b + k * step_b, idesc, k > 0 ? 1u : 0u);
                    umma_commit<false>(sh.empty(ring.stage));
                    ring.next();
                    acc.next();
                }
                if (!ok) {
                    umma_commit<false>(sh.drain());
                    const volatile int no_abort = 0;
                    mbar_wait(sh.drain(), 0, &no_abort, 100000000ull);
                }
            }
        } else {
            // ---------------- scales: two warps, in turn
            const int mine = warp - 2;
            ScaleCopies<COLS, false, BN, Smem::kSlots, 2, 1> copies(sh.scales, sh.scale_full(0), sh.scale_empty(0), lane, mine);
            copies.begin(p, m0, n0, kb0 + mine);
            for (int kb = kb0 + mine; ok && kb < kb1; kb += 2) ok = copies.copy(watch);
            copies.finish();
        }
    } else {
        if (BN == 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;" ::: "memory");
        // ---------------- adding warps: rows 32 * quarter .., every second block
        const int quarter = warp & 3, group = (warp - Smem::kFirst) >> 2;
        float *scratch = sh.scratch + (warp - Smem::kFirst) * 2 * BN;
        const uint32_t taddr0 = tmem + (uint32_t(quarter * 32) << 16);
        using L = Slot<COLS, false>;
        Sums<BN, COLS, false> sums;
        sums.clear();
        if (group == 1) ring.next();
        bool there = false;
        for (int i = group; i < kb1 - kb0; i += 2) {
            auto there_or = [&](int b, bool wait) {
                const uint32_t scales = sh.scale_full(b & 7), full = sh.empty(ring.stage), phase = uint32_t(b >> 3) & 1u;
                return wait ? wait_both(watch, scales, phase, full, ring.phase) : both_there(scales, phase, full, ring.phase);
            };
            if (!there) ok = there_or(i, true);
            if (!ok) break;
            tc_fence_after();
            ring.next();
            ring.next();
            sums.add(
                taddr0 + uint32_t((i & 3) * BN), sh.scales + (i & 7) * L::kFloats, quarter * 32 + lane, 0, scratch, lane,
                [&] { there = i + 2 < kb1 - kb0 && there_or(i + 2, false); },
                [&] {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(sh.acc_empty(i & 3));
                        if (i >= 2) mbar_arrive(sh.scale_empty((i - 2) & 7));  // of the block before
                    }
                });
        }
        // every copy has landed and every MMA of this group has been read; once both groups are here the ring's
        // memory takes the sums, those of the even blocks first
        float *to = sh.sums + (quarter * 32 + lane) * Smem::kRow;
        const bool failed = __any_sync(kFull, !ok);
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
        if (group == 0 && !failed) {
#pragma unroll
            for (int i = 0; i < BN; i += 4)
                *reinterpret_cast<float4 *>(to + i) =
                    make_float4(sums.at[i / 2].x, sums.at[i / 2].y, sums.at[i / 2 + 1].x, sums.at[i / 2 + 1].y);
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
        if (group == 1 && !failed && kb1 - kb0 > 1) {
#pragma unroll
            for (int i = 0; i < BN; i += 4) {
                float4 &v = *reinterpret_cast<float4 *>(to + i);
                v = make_float4(v.x + sums.at[i / 2].x, v.y + sums.at[i / 2].y, v.z + sums.at[i / 2 + 1].x, v.w + sums.at[i / 2 + 1].y);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_free<false>(tmem, Smem::kTmem);
    if (p.splits > 1) cluster_sync();
    if (*sh.abort_flag == 0) {
        if (p.c_type == GEMM_TYPE_F32) store_tile<float, BN>(p, sh.sums, rank, m0, n0);
        else if (p.c_type == GEMM_TYPE_F16) store_tile<__half, BN>(p, sh.sums, rank, m0, n0);
        else store_tile<__nv_bfloat16, BN>(p, sh.sums, rank, m0, n0);
    }
    if (p.splits > 1) {
        __syncwarp();
        cluster_sync();  // the others may still read this CTA's sums
    }
    if (p.tail >= 0) asm volatile("griddepcontrol.wait;" ::: "memory");  // what follows waits for this kernel alone
}

// ------------------------------------------------------------------ host side
// An 8-bit row-major matrix in boxes of 128 bytes x box_rows with the 128-byte swizzle.
bool make_map8(CUtensorMap *map, const void *ptr, int64_t rows, int64_t cols, int64_t ld, int box_rows)
{
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), 1};
    const cuuint64_t strides[2] = {cuuint64_t(ld), cuuint64_t(ld) * cuuint64_t(rows)};
    const cuuint32_t box[3] = {128, cuuint32_t(box_rows), 1}, steps[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(ptr), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool operand_map(CUtensorMap *map, const ScaledOperand &o, int64_t mn, int64_t K, int box_rows)
{
    return o.mn ? make_map8(map, o.at, K, mn, o.ld, 128) : make_map8(map, o.at, mn, K, o.ld, box_rows);
}

ScaledParams params_of(const ScaledArgs &a, int tile_m, int tile_n, unsigned int *status)
{
    ScaledParams p{};
    p.M = a.M;
    p.N = a.N;
    p.num_kb = int((a.K + 127) / 128);
    p.tiles_m = int((a.M + tile_m - 1) / tile_m);
    p.tiles_n = int((a.N + tile_n - 1) / tile_n);
    p.splits = 1;
    p.tail = -1;
    p.a_mn = a.a.mn;
    p.b_mn = a.b.mn;
    p.formats = (a.a.q_type == GEMM_TYPE_E5M2 ? 1u << 7 : 0u) | (a.b.q_type == GEMM_TYPE_E5M2 ? 1u << 10 : 0u);
    p.sa = a.a.scales;
    p.sa_mn = a.a.s_mn;
    p.sa_k = a.a.s_k;
    p.a_shift = a.a.mn_shift;
    p.sb = a.b.scales;
    p.sb_mn = a.b.s_mn;
    p.sb_k = a.b.s_k;
    p.b_shift = a.b.mn_shift;
    p.C = a.C;
    p.ldc = a.ldc;
    p.c_type = a.c_type;
    p.status = status;
    test_hooks(p.timeout_ns, p.inject_stall);
    return p;
}

// tail: of K, for the tiles beyond the last full wave, which single CTAs take then; 0: pairs take all.
template <bool COLS, bool F32>
cudaError_t launch_pairs(const DeviceInfo &dev, const ScaledArgs &a, int tail, unsigned int *status, cudaStream_t stream)
{
    static std::atomic<int> cache[64];
    using Smem = PairSmem<COLS>;
    auto *kernel = scaled_pair_kernel<COLS, F32>;
    const int pairs = resident_pairs(kernel, kPairThreads, Smem::kBytes, dev.device, cache);
    if (pairs <= 0) return cudaErrorInitializationError;
    ScaledParams p = params_of(a, 256, 256, status);
    CUtensorMap ma, mb, mc;
    std::memset(&mc, 0, sizeof(mc));
    if (!operand_map(&ma, a.a, a.M, a.K, 128) || !operand_map(&mb, a.b, a.N, a.K, 128)) return cudaErrorInvalidValue;
    p.c_tma = make_store_map(&mc, a.C, a.c_type, a.M, a.N, a.ldc, 1, 0, true);
    const int64_t tiles = int64_t(p.tiles_m) * p.tiles_n;
    if (tiles >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    const int64_t left = tail > 0 && tiles > pairs ? tiles % pairs : 0;
    p.tiles = int(tiles - left);
    cudaError_t e = launch_chained(kernel, dim3(unsigned(2 * (tiles < pairs ? tiles : pairs))), kPairThreads, Smem::kBytes, 2, stream, ma, mb, mc, p);
    if (e != cudaSuccess || left == 0) return e;
    using Tile = TileSmem<128>;
    auto *rest = scaled_tile_kernel<128, COLS>;
    if ((e = allow_smem_once(rest, Tile::kBytes)) != cudaSuccess) return e;
    p.tail = p.tiles;
    p.splits = tail;
    return launch_chained(rest, dim3(unsigned(4 * left * tail)), Tile::kThreads, Tile::kBytes, tail, stream, ma, mb, p);
}

template <int BN, bool COLS>
cudaError_t launch_tiles(const ScaledArgs &a, int splits, int transposed, unsigned int *status, cudaStream_t stream)
{
    using Smem = TileSmem<BN>;
    auto *kernel = scaled_tile_kernel<BN, COLS>;
    const cudaError_t e = allow_smem_once(kernel, Smem::kBytes);
    if (e != cudaSuccess) return e;
    ScaledParams p = params_of(a, 128, BN, status);
    p.splits = splits;
    p.transposed = transposed;
    CUtensorMap ma, mb;
    if (!operand_map(&ma, a.a, a.M, a.K, 128) || !operand_map(&mb, a.b, a.N, a.K, BN)) return cudaErrorInvalidValue;
    const int64_t ctas = int64_t(p.tiles_m) * p.tiles_n * splits;
    if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    return launch_chained(kernel, dim3(unsigned(ctas)), Smem::kThreads, Smem::kBytes, splits, stream, ma, mb, p);
}

template <int BN>
cudaError_t launch_tiles(const ScaledArgs &a, int splits, int transposed, unsigned int *status, cudaStream_t stream)
{
    return a.b.mn_shift == 0 ? launch_tiles<BN, true>(a, splits, transposed, status, stream)
                             : launch_tiles<BN, false>(a, splits, transposed, status, stream);
}

struct Plan {
    bool pairs, swap;
    int bn, splits;  // splits with pairs: of the tail, 0 without one
};

// The form of least modelled time, in us.  A tile's CTA takes `base` (`swapped` more, to store turned) and `block` a
// K block, the sum of a cluster's parts `join`; CTAs run one an SM.  A pair's tile takes 0.5 a block, 0.72 with
// column scales.  Tiles' copies reach 5.5 TB/s.  Fitted to 35 shapes from 1 x 512 x 512 to 3000 x 4096 x 4096, each
// with up to 16 plans: the plan taken is on average 3% slower than the fastest (64 x 8192 x 4096: 64 columns unsplit
// 10.6, the halves of 128 columns 11.3, swapped 12.7; 1 x 4096 x 4096: swapped, 4 parts 7.0, 2 parts 7.9, unswapped 15.6
// and more).  The tiles beyond the last full wave in single CTAs: 2304 x 2304 x 4096, 5 tiles, 33.5 us with pairs alone,
// 32.4, 30.2 and 29.1 with 1, 2 and 4 parts of K; 8192 x 4096 x 4096, 56 tiles, 110 with pairs alone, 121 and more.
Plan plan_of(const DeviceInfo &dev, const ScaledArgs &a)
{
    struct Form {
        int bn;
        double base, swapped, block, cols, join;
    };
    static constexpr Form kForms[3] = {{32, 3.7, 0.8, 0.20, 0.04, 1.0}, {64, 3.9, 1.3, 0.25, 0.10, 1.7}, {128, 5.2, 2.0, 0.33, 0.06, 2.6}};
    auto up = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
    const int64_t kb = up(a.K, 128);
    const double copies = double(a.M + a.N) * double(a.K) / 5.5e6;
    const int64_t pairs = dev.num_sms / 2;
    Plan best{true, false, 128, 0};
    const int64_t big = up(a.M, 256) * up(a.N, 256), left = big > pairs ? big % pairs : 0;
    const double wave = double(kb) * (a.b.mn_shift == 0 ? 0.72 : 0.5) + 0.3;
    double least = 4.7 + double(up(big, pairs)) * wave;
    for (int splits = 1; left > 0 && splits <= 8 && splits <= kb; splits *= 2) {
        const Form &f = kForms[2];
        const double cost = 4.7 + double(big / pairs) * wave + (splits > 1 ? f.join : 0.0) +
                            double(up(4 * left * splits, dev.num_sms)) * (f.base + double(up(kb, splits)) * (f.block + (a.b.mn_shift == 0 ? f.cols : 0.0)));
        if (cost < least) {
            least = cost;
            best.splits = splits;
        }
    }
    for (int swap = 0; swap < 2; ++swap) {
        const ScaledOperand &b = swap ? a.a : a.b;
        const int64_t m = swap ? a.N : a.M, n = swap ? a.M : a.N;
        for (const Form &f : kForms) {
            if (f.bn < 128 && b.mn) continue;  // an operand stored K x N comes in boxes of 128 columns
            const int64_t tiles = up(m, 128) * up(n, f.bn);
            for (int splits = 1; splits <= 8 && splits <= kb; splits *= 2) {
                const double blocks = double(up(kb, splits)) * (f.block + (b.mn_shift == 0 ? f.cols : 0.0));
                const double waves = double(up(tiles * splits, dev.num_sms));
                const double cost = waves * (f.base + (swap ? f.swapped : 0.0)) + (waves * blocks > copies ? waves * blocks : copies) + (splits > 1 ? f.join : 0.0);
                if (cost < least) {
                    least = cost;
                    best = Plan{false, swap != 0, f.bn, splits};
                }
            }
        }
    }
    // GEMM_GB300_SCALED_PLAN (tests and sweeps): P or P:splits of the tail for pairs, or BN:splits or
    // BN:splits:s (operands swapped)
    if (const char *e = std::getenv("GEMM_GB300_SCALED_PLAN"); e && *e) {
        int bn = 0, splits = 0;
        char s = 0;
        if (*e == 'P') {
            best = Plan{true, false, 128, 0};
            if (std::sscanf(e, "P:%d", &splits) == 1 && (splits == 1 || splits == 2 || splits == 4 || splits == 8)) best.splits = splits;
        } else if (std::sscanf(e, "%d:%d:%c", &bn, &splits, &s) >= 2 && (bn == 32 || bn == 64 || bn == 128) &&
                   (splits == 1 || splits == 2 || splits == 4 || splits == 8) && (bn == 128 || !(s == 's' ? a.a : a.b).mn)) {
            best = Plan{false, s == 's', bn, splits};
        }
    }
    return best;
}

}  // namespace

cudaError_t launch_scaled(const DeviceInfo &dev, const ScaledArgs &a, cudaStream_t stream)
{
    unsigned int *status = device_status_word(dev.device);
    if (status == nullptr) return cudaErrorInitializationError;
    const Plan plan = plan_of(dev, a);
    if (plan.pairs) {
        const bool cols = a.b.mn_shift == 0, f32 = a.c_type == GEMM_TYPE_F32;
        if (cols) return f32 ? launch_pairs<true, true>(dev, a, plan.splits, status, stream) : launch_pairs<true, false>(dev, a, plan.splits, status, stream);
        return f32 ? launch_pairs<false, true>(dev, a, plan.splits, status, stream) : launch_pairs<false, false>(dev, a, plan.splits, status, stream);
    }
    ScaledArgs t = a;
    if (plan.swap) {
        t.M = a.N;
        t.N = a.M;
        t.a = a.b;
        t.b = a.a;
    }
    if (plan.bn == 32) return launch_tiles<32>(t, plan.splits, plan.swap, status, stream);
    if (plan.bn == 64) return launch_tiles<64>(t, plan.splits, plan.swap, status, stream);
    return launch_tiles<128>(t, plan.splits, plan.swap, status, stream);
}

}  // namespace gemm
