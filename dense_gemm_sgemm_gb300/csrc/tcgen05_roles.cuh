// What the roles of the tcgen05 kernels share beside the PTX wrappers: bounded waits that report, ring
// positions, accumulator hand-over, staged TMA stores, 16-bit packing.
#pragma once

#include <atomic>
#include <cstdlib>

#include "gemm_internal.h"
#include "routed_internal.h"
#include "tcgen05_ptx.cuh"
#include "tensor_map.h"

namespace gemm {

// The waits' limit and where they report.
struct Watch {
    volatile int *abort_flag;
    unsigned int *status;
    uint64_t timeout_ns;
    __device__ __forceinline__ void raise() const
    {
        *abort_flag = 1;
        atomicOr(status, 1u);
    }
    template <bool CLUSTER = false> __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const
    {
        if (mbar_wait<CLUSTER>(bar, parity, abort_flag, timeout_ns)) return true;
        raise();
        return false;
    }
};

// OR of `pred` over WARPS epilogue warps (named barrier 1), which all call it.
template <int WARPS> __device__ __forceinline__ bool epilogue_any(bool pred)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(static_cast<uint32_t>(pred)), "n"(32 * WARPS)
                 : "memory");
    return r != 0;
}

__device__ __forceinline__ uint16_t to_16(float v, bool bf16)
{
    return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

__device__ __forceinline__ uint32_t pack_16(float lo, float hi, bool bf16)
{
    if (bf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Ring position of a role: stage and the parity its next phase completes.
struct Ring {
    int stages, stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ explicit Ring(int n) : stages(n) {}
    __device__ __forceinline__ void next()
    {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// Arrives on the barrier at this address in both CTAs of the pair once the MMAs issued so far have
// completed.
__device__ __forceinline__ void commit_both(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"(uint16_t(3))
                 : "memory");
}

// The warp has its accumulator columns in registers: one arrival on the issuer's barrier, which may be
// the peer's.  Released at CTA scope only: a release at cluster scope would wait for the warp's global
// stores (the weight gradient of 32 groups of 64 rows, 2048 x 1024, took 57 us with such an arrival
// after the stores, 47 with this one before them).
__device__ __forceinline__ void release_accumulator(uint32_t bar_cluster, int lane)
{
    tc_fence_before();
    __syncwarp();
    if (lane == 0) asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// The epilogue warps' staging tiles and their TMA stores in flight: fp32 pieces fill a tile, 16-bit
// pieces take its halves in turn.
template <bool F32> struct Staging {
    uint8_t *tile;
    int lane, half = 0;
    __device__ __forceinline__ Staging(uint8_t *t, int l) : tile(t), lane(l) {}
    // The place of the next piece, once the store that last read it has done so.
    __device__ __forceinline__ uint8_t *next()
    {
        if (lane == 0) {
            if (F32) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            else asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        }
        __syncwarp();
        half ^= F32 ? 0 : 2048;
        return tile + half;
    }
    // The whole tile, free of stores.
    __device__ __forceinline__ uint8_t *all() const
    {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
        return tile;
    }
    __device__ __forceinline__ void store(const CUtensorMap *map, const uint8_t *piece, int c0, int c1, int c2) const
    {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(map, smem_u32(piece), c0, c1, c2);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
    }
    // Every store has been written; to be called before the CTA ends.
    __device__ __forceinline__ void finish() const
    {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
};

// This lane's row m0 + lane, 32 columns from n0, of C (M x N): through the staging tile to a TMA store of a
// 32 x 32 box (map: make_store_map, swizzled), or where TMA cannot store to 16-byte pieces of rows.  C 16-byte
// aligned, ld a multiple of 8 elements; plane: the matrix of the map's stack, which C points to.
// TRANSPOSED: this lane's column n0 + lane, 32 rows from m0.
template <bool F32, bool TRANSPOSED = false>
__device__ __forceinline__ void store_rows(Staging<F32> &staging, const float (&v)[32], const CUtensorMap *map, bool tma, void *C,
                                           int64_t ld, int64_t m0, int64_t n0, int64_t M, int64_t N, bool bf16, int plane)
{
    const int lane = staging.lane;
    uint8_t *piece = tma ? staging.next() : staging.all();
    uint4 *row = reinterpret_cast<uint4 *>(piece) + lane * (F32 ? 8 : 4);
    if (TRANSPOSED && F32) {
        float *t = reinterpret_cast<float *>(piece) + (lane & 3);
#pragma unroll
        for (int i = 0; i < 32; ++i) t[i * 32 + 4 * ((lane >> 2) ^ (i & 7))] = v[i];
    } else if (TRANSPOSED) {
        uint16_t *t = reinterpret_cast<uint16_t *>(piece) + (lane & 7);
#pragma unroll
        for (int i = 0; i < 32; ++i) t[i * 32 + 8 * ((lane >> 3) ^ ((i >> 1) & 3))] = to_16(v[i], bf16);
    } else if (F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            row[j ^ (lane & 7)] = make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
                                             __float_as_uint(v[4 * j + 3]));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            row[j ^ ((lane >> 1) & 3)] = make_uint4(pack_16(v[8 * j], v[8 * j + 1], bf16), pack_16(v[8 * j + 2], v[8 * j + 3], bf16),
                                                    pack_16(v[8 * j + 4], v[8 * j + 5], bf16), pack_16(v[8 * j + 6], v[8 * j + 7], bf16));
    }
    if (tma) {
        staging.store(map, piece, int(n0), int(m0), plane);
        return;
    }
    __syncwarp();
    constexpr int kPieces = F32 ? 8 : 4, kEach = 32 / kPieces;  // 16-byte pieces of a row, their elements
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int r = i * (32 / kPieces) + lane / kPieces, q = lane % kPieces;
        const int64_t m = m0 + r, n = n0 + q * kEach;
        const uint4 u = reinterpret_cast<const uint4 *>(piece)[r * kPieces + (F32 ? q ^ (r & 7) : q ^ ((r >> 1) & 3))];
        if (m >= M || n >= N) continue;
        uint8_t *dst = static_cast<uint8_t *>(C) + (m * ld + n) * (F32 ? 4 : 2);
        if (n + kEach <= N) {
            *reinterpret_cast<uint4 *>(dst) = u;
        } else {
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < kEach; ++j)
                if (n + j < N) {
                    if (F32) reinterpret_cast<uint32_t *>(dst)[j] = w[j % 4];
                    else reinterpret_cast<uint16_t *>(dst)[j] = uint16_t(w[j / 2] >> (16 * (j & 1)));
                }
        }
    }
    __syncwarp();
}

// A stack of `count` row-major matrices stored to in boxes of 32 x 32.  False where TMA cannot: a box cut
// by the right edge is written in whole 16-byte pieces, so the rows must end on one.
inline bool make_store_map(CUtensorMap *map, void *ptr, int type, int64_t rows, int64_t cols, int64_t ld, int64_t count, int64_t stride,
                    bool swizzled)
{
    auto fn = tensor_map_encoder();
    const bool f32 = type == GEMM_TYPE_F32;
    const int size = f32 ? 4 : 2;
    if (fn == nullptr || cols * size % 16 != 0 || reinterpret_cast<uintptr_t>(ptr) % 16 != 0) return false;
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(count)};
    const cuuint64_t strides[2] = {cuuint64_t(ld) * size, cuuint64_t(count > 1 ? stride : rows * ld) * size};
    const cuuint32_t box[3] = {32, 32, 1};
    const cuuint32_t steps[3] = {1, 1, 1};
    return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : type == GEMM_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                                 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
              3, ptr, dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
              !swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE : f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Two-CTA clusters of `kernel` that can be resident at once; 0 on failure.  `cache`: of this kernel.
template <class K> int resident_pairs(K *kernel, int threads, int smem, int dev, std::atomic<int> (&cache)[64])
{
    const int known = cache[dev & 63].load(std::memory_order_acquire);
    if (known > 0) return known;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    cache[dev & 63].store(n, std::memory_order_release);
    return n;
}

// GEMM_GB300_TEST_INJECT_STALL: a producer never fills its first slice, and waits are short.
inline void test_hooks(uint64_t &timeout_ns, int &inject_stall)
{
    timeout_ns = 2000000000ull;
    inject_stall = 0;
    if (const char *e = std::getenv("GEMM_GB300_TEST_INJECT_STALL"); e && e[0] == '1') {
        inject_stall = 1;
        timeout_ns = 20000000ull;
    }
}

}  // namespace gemm
