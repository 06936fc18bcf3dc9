// What the tcgen05 translation units share on the host side.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

namespace gemm {

// The driver's tensor-map encoder, looked up once (NULL without a driver).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Device address, on the current device `dev`, of the error word that kernels raise when a bounded
// wait expires (NULL on failure).
unsigned int *device_status_word(int dev);

}  // namespace gemm
