// Declarations of the orthogonalised update.  The launchers take validated arguments (orthogonal.cu).
#pragma once

#include "routed_internal.h"

namespace gemm {

// n <= k: sides of the matrices as the products take them; a matrix with more rows than columns is taken
// transposed.  Matrices of the call's work space, `count` of each, rows on whole 128-byte lines:
//   X     fp16 parts high and low (n x k each), two sets that the steps write in turn
//   E     off-diagonal part of X X^T, parts high and low (n x n each), zeros on the diagonal
//   F     off-diagonal part of b A + c A^2, likewise
//   d, f  the two diagonals in fp32 (n each)
struct OrthogonalLayout {
    int64_t n, k, count, ldk, ldn;
    int64_t x[2], e, f, dd, df, unit, partial;  // byte offsets; unit: 1 / c of each matrix (Norm); partial sums
    int64_t bytes;
};
constexpr int kNormBlocks = 304;  // at most, of a matrix's sum of squares
OrthogonalLayout orthogonal_layout(int64_t count, int64_t rows, int64_t cols);

struct OrthogonalArgs {
    int type, y_type;
    int64_t count, rows, cols;
    const void *G;
    int64_t ldg, strideg;
    void *Y;
    int64_t ldy, stridey;
    float eps;
    void *work;
};
// ||G|| and the parts of G * 2^(kFirstScale - e), 2^e <= ||G|| + eps < 2^(e + 1): |elements| <= 2^15.
constexpr int kFirstScale = 14;
cudaError_t launch_normalise(const OrthogonalArgs &a, const OrthogonalLayout &l, cudaStream_t stream);

// A step X' = (a + b A + c A^2) X, A = X X^T.  x_scale, e_scale, f_scale, next_scale: the powers of two by
// which the parts in memory are larger than what they stand for.
struct OrthogonalStep {
    float a, b, c;
    float x_scale, e_scale, f_scale, next_scale;
};
// The first step's X in memory is to be multiplied by 1 / c of its matrix (unit), the last one writes Y.
cudaError_t launch_orthogonal_steps(const DeviceInfo &dev, const OrthogonalArgs &a, const OrthogonalLayout &l, const OrthogonalStep *plan,
                                    int steps, cudaStream_t stream);

}  // namespace gemm
