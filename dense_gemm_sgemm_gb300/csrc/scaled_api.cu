// Host side of the block-scaled products' C entry points: argument checks, then the launchers.
#include <cuda_runtime.h>

#include "scaled_internal.h"

namespace gemm {
namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 30) - 1;
constexpr int64_t kMaxLd = int64_t(1) << 35;
constexpr int64_t kMaxStride = int64_t(1) << 40;

bool is_type(int t) { return t == GEMM_TYPE_F32 || t == GEMM_TYPE_F16 || t == GEMM_TYPE_BF16; }
bool is_type8(int t) { return t == GEMM_TYPE_E4M3 || t == GEMM_TYPE_E5M2; }
int size_of(int t) { return t == GEMM_TYPE_F32 ? 4 : 2; }
bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool bytes16(const void *p, int64_t ld) { return aligned(p, 16) && ld % 16 == 0; }
gemm_status_t from_cuda(cudaError_t e)
{
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}
gemm_status_t usable(DeviceInfo &dev)
{
    return current_device(dev) && dev.cc_major == 10 && dev.cc_minor == 3 ? GEMM_OK : GEMM_ERR_NO_DEVICE;
}
bool ld_ok(int64_t ld, int64_t cols) { return ld >= (cols > 1 ? cols : 1); }

gemm_status_t check_matrix(int64_t rows, int64_t cols, int64_t ld)
{
    if (rows < 0 || cols < 0 || !ld_ok(ld, cols)) return GEMM_ERR_INVALID_VALUE;
    return rows > kMaxDim || cols > kMaxDim || ld > kMaxLd ? GEMM_ERR_UNSUPPORTED : GEMM_OK;
}
gemm_status_t check_scales(const float *s, int64_t s_row, int64_t s_col)
{
    if (s == nullptr || s_row < 0 || s_col < 0) return GEMM_ERR_INVALID_VALUE;
    if (s_row > kMaxStride || s_col > kMaxStride) return GEMM_ERR_UNSUPPORTED;
    return aligned(s, 4) ? GEMM_OK : GEMM_ERR_MISALIGNED;
}
bool block_ok(int rows, int cols)
{
    return (rows == 1 || rows == 128) && (cols == 1 || cols == 128) && rows + cols > 2;
}
int shift_of(int block) { return block == 128 ? 7 : 0; }

gemm_status_t quantize(gemm_type_t type, gemm_type_t q_type, const QuantizeArgs &a, cudaStream_t stream)
{
    if (!is_type(type) || !is_type8(q_type)) return GEMM_ERR_INVALID_VALUE;
    gemm_status_t s = check_matrix(a.rows, a.cols, a.ldx);
    if (s != GEMM_OK) return s;
    const bool rows = a.Q != nullptr || a.s.at != nullptr, columns = a.Qc != nullptr || a.sc.at != nullptr;
    if ((rows && (s = check_matrix(a.rows, a.cols, a.ldq)) != GEMM_OK) ||
        (columns && (s = check_matrix(a.rows, a.cols, a.ldqc)) != GEMM_OK))
        return s;
    if (a.rows == 0 || a.cols == 0) return GEMM_OK;
    if (a.X == nullptr || (rows && a.Q == nullptr) || (columns && a.Qc == nullptr) || (!rows && !columns)) return GEMM_ERR_INVALID_VALUE;
    if ((rows && (s = check_scales(a.s.at, a.s.row, a.s.col)) != GEMM_OK) ||
        (columns && (s = check_scales(a.sc.at, a.sc.row, a.sc.col)) != GEMM_OK))
        return s;
    if (!aligned(a.X, size_of(type)) || (rows && !bytes16(a.Q, a.ldq)) || (columns && !bytes16(a.Qc, a.ldqc)))
        return GEMM_ERR_MISALIGNED;
    DeviceInfo dev;
    if ((s = usable(dev)) != GEMM_OK) return s;
    return from_cuda(launch_quantize(a, stream));
}

}  // namespace
}  // namespace gemm

using namespace gemm;

extern "C" {

gemm_status_t gemm_quantize_blocks(gemm_type_t type, gemm_type_t q_type, int64_t rows, int64_t cols, const void *X, int64_t ldx,
                                   int block_rows, int block_cols, void *Q, int64_t ldq, float *scales, int64_t s_row,
                                   int64_t s_col, void *stream)
{
    if (!block_ok(block_rows, block_cols)) return GEMM_ERR_INVALID_VALUE;
    if (rows > 0 && cols > 0 && (Q == nullptr || scales == nullptr)) return GEMM_ERR_INVALID_VALUE;
    QuantizeArgs a{type, q_type, rows, cols, X, ldx, nullptr, 0, Scales{}, nullptr, 0, Scales{}};
    const Scales s{scales, s_row, s_col, shift_of(block_rows), shift_of(block_cols)};
    if (block_cols == 1) {
        a.Qc = Q;
        a.ldqc = ldq;
        a.sc = s;
    } else {
        a.Q = Q;
        a.ldq = ldq;
        a.s = s;
    }
    return quantize(type, q_type, a, static_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_quantize_both(gemm_type_t type, gemm_type_t q_type, int64_t rows, int64_t cols, const void *X, int64_t ldx,
                                 void *Q, int64_t ldq, float *scales, int64_t s_row, int64_t s_col, void *Qc, int64_t ldqc,
                                 float *scales_c, int64_t sc_row, int64_t sc_col, void *stream)
{
    if (rows > 0 && cols > 0 && (Q == nullptr || scales == nullptr || Qc == nullptr || scales_c == nullptr))
        return GEMM_ERR_INVALID_VALUE;
    const QuantizeArgs a{type, q_type, rows, cols, X, ldx, Q, ldq, Scales{scales, s_row, s_col, 0, 7},
                         Qc, ldqc, Scales{scales_c, sc_row, sc_col, 7, 0}};
    return quantize(type, q_type, a, static_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_dequantize_blocks(gemm_type_t q_type, gemm_type_t y_type, int64_t rows, int64_t cols, const void *Q,
                                     int64_t ldq, int block_rows, int block_cols, const float *scales, int64_t s_row,
                                     int64_t s_col, void *Y, int64_t ldy, void *stream)
{
    if (!is_type(y_type) || !is_type8(q_type) || !block_ok(block_rows, block_cols)) return GEMM_ERR_INVALID_VALUE;
    gemm_status_t s;
    if ((s = check_matrix(rows, cols, ldq)) != GEMM_OK || (s = check_matrix(rows, cols, ldy)) != GEMM_OK) return s;
    if (rows == 0 || cols == 0) return GEMM_OK;
    if (Q == nullptr || Y == nullptr) return GEMM_ERR_INVALID_VALUE;
    if ((s = check_scales(scales, s_row, s_col)) != GEMM_OK) return s;
    if (!bytes16(Q, ldq) || !aligned(Y, size_of(y_type))) return GEMM_ERR_MISALIGNED;
    DeviceInfo dev;
    if ((s = usable(dev)) != GEMM_OK) return s;
    const Scales at{const_cast<float *>(scales), s_row, s_col, shift_of(block_rows), shift_of(block_cols)};
    return from_cuda(launch_dequantize(q_type, y_type, rows, cols, Q, ldq, at, Y, ldy, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_scaled_matmul(gemm_type_t a_type, gemm_type_t b_type, gemm_type_t c_type, gemm_op_t opA, gemm_op_t opB, int64_t M,
                                 int64_t N, int64_t K, const void *A, int64_t lda, int a_block, const float *a_scales,
                                 int64_t sa_row, int64_t sa_col, const void *B, int64_t ldb, int b_block, const float *b_scales,
                                 int64_t sb_row, int64_t sb_col, void *C, int64_t ldc, void *stream)
{
    if (!is_type8(a_type) || !is_type8(b_type) || !is_type(c_type) || (opA != GEMM_OP_N && opA != GEMM_OP_T) ||
        (opB != GEMM_OP_N && opB != GEMM_OP_T) || (a_block != 1 && a_block != 128) || (b_block != 1 && b_block != 128))
        return GEMM_ERR_INVALID_VALUE;
    gemm_status_t s;
    if ((s = check_matrix(opA == GEMM_OP_N ? M : K, opA == GEMM_OP_N ? K : M, lda)) != GEMM_OK ||
        (s = check_matrix(opB == GEMM_OP_N ? K : N, opB == GEMM_OP_N ? N : K, ldb)) != GEMM_OK ||
        (s = check_matrix(M, N, ldc)) != GEMM_OK)
        return s;
    if (M == 0 || N == 0) return GEMM_OK;
    if (C == nullptr || (K > 0 && (A == nullptr || B == nullptr))) return GEMM_ERR_INVALID_VALUE;
    if (K > 0 && ((s = check_scales(a_scales, sa_row, sa_col)) != GEMM_OK || (s = check_scales(b_scales, sb_row, sb_col)) != GEMM_OK))
        return s;
    if ((K > 0 && (!bytes16(A, lda) || !bytes16(B, ldb))) || !aligned(C, 16) || ldc % 8 != 0) return GEMM_ERR_MISALIGNED;
    DeviceInfo dev;
    if ((s = usable(dev)) != GEMM_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (K == 0)
        return from_cuda(cudaMemset2DAsync(C, size_t(ldc) * size_of(c_type), 0, size_t(N) * size_of(c_type), size_t(M), st));
    // the kernels take both operands by rows of the result and K
    const ScaledOperand a{a_type, opA == GEMM_OP_T, A, lda, a_scales, opA == GEMM_OP_T ? sa_col : sa_row,
                          opA == GEMM_OP_T ? sa_row : sa_col, shift_of(a_block)};
    const ScaledOperand b{b_type, opB == GEMM_OP_N, B, ldb, b_scales, opB == GEMM_OP_N ? sb_col : sb_row,
                          opB == GEMM_OP_N ? sb_row : sb_col, shift_of(b_block)};
    return from_cuda(launch_scaled(dev, ScaledArgs{M, N, K, a, b, c_type, C, ldc}, st));
}

}  // extern "C"
