// Declarations of the block-scaled 8-bit matrices and their products.  The launchers take validated
// arguments (scaled_api.cu).
#pragma once

#include <cuda_fp8.h>

#include "routed_internal.h"

namespace gemm {

// An 8-bit matrix's scales: the scale of element (i, j) is at[(i >> row_shift) * row + (j >> col_shift) * col].
struct Scales {
    float *at;
    int64_t row, col;
    int row_shift, col_shift;
};

struct QuantizeArgs {
    int type, q_type;
    int64_t rows, cols;
    const void *X;
    int64_t ldx;
    // blocks of 1 x 128 or 128 x 128 elements (or NULL), and of 128 x 1 (or NULL)
    void *Q;
    int64_t ldq;
    Scales s;
    void *Qc;
    int64_t ldqc;
    Scales sc;
};
cudaError_t launch_quantize(const QuantizeArgs &a, cudaStream_t stream);
cudaError_t launch_dequantize(int q_type, int y_type, int64_t rows, int64_t cols, const void *Q, int64_t ldq, const Scales &s, void *Y,
                              int64_t ldy, cudaStream_t stream);

// C (M x N) = A B^T over K in blocks of 128: `mn` tells that the operand is stored K x M (K x N), and
// scales are by its rows M (N) and K blocks.
struct ScaledOperand {
    int q_type, mn;
    const void *at;
    int64_t ld;
    const float *scales;
    int64_t s_mn, s_k;
    int mn_shift;  // 0: a scale for every row, 7: for every 128
};
struct ScaledArgs {
    int64_t M, N, K;
    ScaledOperand a, b;
    int c_type;
    void *C;
    int64_t ldc;
};
cudaError_t launch_scaled(const DeviceInfo &dev, const ScaledArgs &a, cudaStream_t stream);

}  // namespace gemm
