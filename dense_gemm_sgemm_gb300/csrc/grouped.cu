// Grouped products: which kernel takes which call.
#include <cuda_runtime.h>

#include "routed_internal.h"

namespace gemm {

gemm_status_t launch_grouped(const DeviceInfo &dev, const GroupedArgs &a, cudaStream_t stream)
{
    const int64_t groups = a.y_rows < a.groups ? a.y_rows : a.groups;  // at most that many have rows
    const bool few = a.opW == GEMM_OP_T && a.y_rows <= 16 * groups;
    cudaError_t e;
    if (few || a.K == 0 || a.x_rows == 0) e = launch_few_rows(dev, a, stream);
    else e = launch_many_rows(dev, a, stream);
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace gemm
