// Grouped products: which kernel takes which call.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdlib>

#include "routed_internal.h"

namespace gemm {

namespace {
// Sets a function attribute of a kernel on the current device unless `done` holds that it was set.
// Open addressing over a fixed table, several times the number of kernels: no allocation, so no
// exception can leave a C entry point.
constexpr int kSlots = 512;
cudaError_t set_once(std::atomic<uintptr_t> (&done)[kSlots], const void *kernel, cudaFuncAttribute attribute, int value)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    // host functions start on 16-byte boundaries at least: the device number takes the low bits
    const uintptr_t key = reinterpret_cast<uintptr_t>(kernel) * 4 + uintptr_t(dev & 63);
    for (int i = 0; i < kSlots; ++i) {
        std::atomic<uintptr_t> &slot = done[(key / 64 + key % 64 + uintptr_t(i)) % kSlots];
        uintptr_t held = slot.load(std::memory_order_acquire);
        if (held == key) return cudaSuccess;
        if (held != 0) continue;
        e = cudaFuncSetAttribute(kernel, attribute, value);
        if (e == cudaSuccess) slot.compare_exchange_strong(held, key, std::memory_order_acq_rel);
        return e;
    }
    return cudaFuncSetAttribute(kernel, attribute, value);
}
}  // namespace

cudaError_t allow_smem_once(const void *kernel, int bytes)
{
    static std::atomic<uintptr_t> done[kSlots];
    return set_once(done, kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

cudaError_t allow_large_cluster_once(const void *kernel)
{
    static std::atomic<uintptr_t> done[kSlots];
    return set_once(done, kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

// The few-rows kernel takes the calls that leave the tcgen05 kernel's pairs of SMs without tiles.
// Both read every weight once from memory; measured, 8 of 64 experts of 2048 x 1024, gated product,
// us few / many: 1 token 17.5 / 18.0, 4 tokens 43 / 42, 16 tokens 85 / 77, and with 128 experts
// 64 tokens 200 / 170, 512 tokens 445 / 186.  One matrix of 4096 x 4096 with adapters: 24 tokens
// 12 / 16, 64 tokens 21 / 28, 80 tokens 32 / 28, 128 tokens 34 / 29.
bool takes_few_rows(const DeviceInfo &dev, const GroupedArgs &a)
{
    if (a.K == 0) return true;
    if (a.opW != GEMM_OP_T) return false;
    const int64_t groups = a.y_rows < a.groups ? a.y_rows : a.groups;  // at most that many have rows
    // GEMM_GB300_GROUPED_FEW=n (sweeps only): the few-rows kernel up to n rows a group
    if (const char *v = std::getenv("GEMM_GB300_GROUPED_FEW"); v && v[0]) return a.y_rows <= std::atoi(v) * groups;
    const int64_t features = a.gated ? 128 : 256;
    return a.y_rows <= 64 && groups * ((a.N + features - 1) / features) < dev.num_sms / 2;
}

gemm_status_t launch_grouped(const DeviceInfo &dev, const GroupedArgs &call, cudaStream_t stream)
{
    GroupedArgs a = call;
    if (a.x_rows == 0) a.K = 0;  // every row is outside X: zeros, and W is not read
    const int64_t groups = a.y_rows < a.groups ? a.y_rows : a.groups;
    cudaError_t e = cudaSuccess;
    if (takes_few_rows(dev, a)) {
        e = launch_few_rows(dev, a, stream);
    } else {
        // Gathered rows: TMA takes 82 cycles for four of them, as long as the MMAs of a slice of 160
        // tokens, where a box of 128 contiguous rows costs next to nothing.  So large groups pay for
        // laying the rows out first (64 groups of 512 rows, 2 x 1024 x 2048 gated: gathered 617 us,
        // contiguous 206 us and the copy), small ones gather.
        if (a.rows != nullptr && a.work != nullptr && a.y_rows > 64 * groups) {
            const int64_t ld = (a.K + 63) / 64 * 64;  // whole 128-byte lines, as the copies read them
            e = launch_gather(a, a.work, ld, stream);
            a.X = a.work;
            a.ldx = ld;
            a.x_rows = a.y_rows;
            a.rows = nullptr;
        }
        if (e == cudaSuccess) e = launch_many_rows(dev, a, stream);
    }
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace gemm
