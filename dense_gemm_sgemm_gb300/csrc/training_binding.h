// Python binding of the block-scaled 8-bit products (see scaled.py) and of the orthogonalised update (see
// update.py); included by routed_binding.cpp, whose helpers it uses.

gemm_type_t type8_of(at::ScalarType t, const char *what)
{
    TORCH_CHECK_TYPE(t == at::kFloat8_e4m3fn || t == at::kFloat8_e5m2, what, ": float8_e4m3fn or float8_e5m2 wanted, got ", t);
    return t == at::kFloat8_e4m3fn ? GEMM_TYPE_E4M3 : GEMM_TYPE_E5M2;
}

// These calls record no gradient: a tensor that would have one is refused rather than its gradient dropped in silence.
const at::Tensor &constant(const at::Tensor &t, const char *what)
{
    TORCH_CHECK_VALUE(!(t.requires_grad() && c10::GradMode::is_enabled()), what,
                      ": requires a gradient, which this call does not record (torch.no_grad() takes its value)");
    return t;
}

int64_t blocks_of(int64_t size) { return (size + 127) / 128; }

// An 8-bit matrix: as matrix(), rows on 16-byte pieces being 16 elements.
Matrix matrix8(Device &device, PyObject *o, const char *what)
{
    Matrix m = matrix(device, o, what);
    constant(m.t, what);
    if (m.rows <= 1) m.ld = std::max((m.cols + 15) & ~int64_t(15), int64_t(16));
    return m;
}

// The scales of an 8-bit matrix, one for every `rows` x `cols` elements, which their count along each axis tells.
struct BlockScales {
    float *at;
    int64_t row, col;
    int rows, cols;
};
int block_along(int64_t count, int64_t size, const char *what)
{
    if (count == blocks_of(size)) return 128;
    TORCH_CHECK_VALUE(count == size, what, ": ", size, " or ", blocks_of(size), " along an axis of ", size, " elements wanted, got ", count);
    return 1;
}
BlockScales scales_of(Device &device, PyObject *o, const Matrix &q, const char *what)
{
    const at::Tensor &t = constant(tensor(device, o, what), what);
    same_type(t, at::kFloat, what);
    TORCH_CHECK_VALUE(t.dim() == 2, what, ": 2-D wanted");
    return BlockScales{t.data_ptr<float>(), t.stride(0), t.stride(1), block_along(t.size(0), q.rows, what),
                       block_along(t.size(1), q.cols, what)};
}

// New memory of given strides (without the dispatcher's views: they cost a microsecond each).
at::Tensor strided(at::IntArrayRef shape, at::IntArrayRef strides, at::ScalarType type, const at::Tensor &like)
{
    return at::Tensor(at::detail::empty_strided_cuda(shape, strides, type, like.device()));
}

// New 8-bit memory with rows on 16-byte pieces, and new scales for blocks of rows x cols: those of 1 x 128
// with the rows next to one another, as the products read them.
struct Quantized {
    at::Tensor q, s;
    int64_t ld;
    Quantized(const Matrix &x, int rows, int cols, at::ScalarType type)
    {
        ld = std::max((x.cols + 15) & ~int64_t(15), int64_t(16));
        q = ld == x.cols ? fresh({x.rows, ld}, type, x.t) : strided({x.rows, x.cols}, {ld, 1}, type, x.t);
        const int64_t across = cols == 1 ? x.cols : blocks_of(x.cols), down = rows == 1 ? x.rows : blocks_of(x.rows);
        s = rows == 1 ? strided({down, across}, {1, std::max(down, int64_t(1))}, at::kFloat, x.t) : fresh({down, across}, at::kFloat, x.t);
    }
};

// x, block_rows, block_cols, dtype, stream
BOUND(quantize_blocks, 5)
    const Matrix x = matrix(device, a[0], "x");
    constant(x.t, "x");
    const Stream stream(a[4], x.t);
    const int rows = small(a[1]), cols = small(a[2]);
    const gemm_type_t type = type_of(x.t.scalar_type(), "x");
    const at::ScalarType dtype = dtype_of(a[3], at::kFloat8_e4m3fn);
    const gemm_type_t q_type = type8_of(dtype, "dtype");
    Quantized out(x, rows, cols, dtype);
    call("gemm_quantize_blocks", [&] {
        return gemm_quantize_blocks(type, q_type, x.rows, x.cols, x.data(), x.ld, rows, cols, out.q.data_ptr(), out.ld,
                                    out.s.data_ptr<float>(), out.s.stride(0), out.s.stride(1), stream.handle);
    });
    return tuple(out.q, out.s);
END_BOUND

// x, dtype, stream
BOUND(quantize_both, 3)
    const Matrix x = matrix(device, a[0], "x");
    constant(x.t, "x");
    const Stream stream(a[2], x.t);
    const gemm_type_t type = type_of(x.t.scalar_type(), "x");
    const at::ScalarType dtype = dtype_of(a[1], at::kFloat8_e4m3fn);
    const gemm_type_t q_type = type8_of(dtype, "dtype");
    Quantized rows(x, 1, 128, dtype), columns(x, 128, 1, dtype);
    call("gemm_quantize_both", [&] {
        return gemm_quantize_both(type, q_type, x.rows, x.cols, x.data(), x.ld, rows.q.data_ptr(), rows.ld, rows.s.data_ptr<float>(),
                                  rows.s.stride(0), rows.s.stride(1), columns.q.data_ptr(), columns.ld, columns.s.data_ptr<float>(),
                                  columns.s.stride(0), columns.s.stride(1), stream.handle);
    });
    return tuple(rows.q, rows.s, columns.q, columns.s);
END_BOUND

// q, scales, out_dtype, stream
BOUND(dequantize_blocks, 4)
    const Matrix q = matrix8(device, a[0], "q");
    const Stream stream(a[3], q.t);
    const gemm_type_t q_type = type8_of(q.t.scalar_type(), "q");
    const BlockScales s = scales_of(device, a[1], q, "scales");
    TORCH_CHECK_VALUE(s.rows == 128 || s.cols == 128, "scales: one for every element");
    const at::ScalarType dtype = dtype_of(a[2], at::kBFloat16);
    const gemm_type_t y_type = type_of(dtype, "out_dtype");
    Padded y = padded(q.rows, q.cols, dtype, q.t);
    call("gemm_dequantize_blocks", [&] {
        return gemm_dequantize_blocks(q_type, y_type, q.rows, q.cols, q.data(), q.ld, s.rows, s.cols, s.at, s.row, s.col,
                                      y.t.data_ptr(), std::max(y.ld, int64_t(8)), stream.handle);
    });
    return wrap(y.t);
END_BOUND

// A, A_scales, B, B_scales, opA, opB, out_dtype, stream
BOUND(scaled_matmul, 8)
    const Matrix A = matrix8(device, a[0], "A"), B = matrix8(device, a[2], "B");
    const Stream stream(a[7], A.t);
    const auto opA = static_cast<gemm_op_t>(small(a[4])), opB = static_cast<gemm_op_t>(small(a[5]));
    const gemm_type_t a_type = type8_of(A.t.scalar_type(), "A"), b_type = type8_of(B.t.scalar_type(), "B");
    const BlockScales sa = scales_of(device, a[1], A, "A_scales"), sb = scales_of(device, a[3], B, "B_scales");
    const bool at_ = opA == GEMM_OP_T, bn = opB == GEMM_OP_N;
    const int64_t M = at_ ? A.cols : A.rows, K = at_ ? A.rows : A.cols, N = bn ? B.cols : B.rows;
    same(bn ? B.rows : B.cols, K, "inner dimension of B");
    TORCH_CHECK_VALUE(K <= 1 || ((at_ ? sa.rows : sa.cols) == 128 && (bn ? sb.rows : sb.cols) == 128),
                      "scales: one for every 128 elements of the inner dimension wanted");
    const at::ScalarType dtype = dtype_of(a[6], at::kBFloat16);
    const gemm_type_t c_type = type_of(dtype, "out_dtype");
    Padded C = padded(M, N, dtype, A.t);
    call("gemm_scaled_matmul", [&] {
        return gemm_scaled_matmul(a_type, b_type, c_type, opA, opB, M, N, K, A.data(), A.ld, at_ ? sa.cols : sa.rows, sa.at, sa.row,
                                  sa.col, B.data(), B.ld, bn ? sb.cols : sb.rows, sb.at, sb.row, sb.col, C.t.data_ptr(), std::max(C.ld, int64_t(8)),
                                  stream.handle);
    });
    return wrap(C.t);
END_BOUND

// g, steps, coefficients (a tuple of 3 * steps numbers), eps, out_dtype, stream
BOUND(orthogonalize, 6)
    const at::Tensor &t = constant(tensor(device, a[0], "g"), "g");
    TORCH_CHECK_VALUE(t.dim() == 2 || t.dim() == 3, "g: a matrix or a stack of matrices (2-D or 3-D) wanted");
    const Matrix x = matrix(device, a[0], "g", int(t.dim()));
    const Stream stream(a[5], t);
    const gemm_type_t type = type_of(t.scalar_type(), "g");
    const int steps = small(a[1]);
    TORCH_CHECK_VALUE(PyTuple_Check(a[2]) && PyTuple_GET_SIZE(a[2]) <= 3 * 64 && PyTuple_GET_SIZE(a[2]) == 3 * Py_ssize_t(steps),
                      "coefficients: three for each of 1 to 64 steps wanted");
    float coefficients[3 * 64];
    for (int i = 0; i < 3 * steps; ++i) coefficients[i] = real(PyTuple_GET_ITEM(a[2], i));
    const float eps = real(a[3]);
    const at::ScalarType dtype = dtype_of(a[4], at::kBFloat16);
    const gemm_type_t y_type = type_of(dtype, "out_dtype");
    const int64_t count = t.dim() == 3 ? t.size(0) : 1, stride = t.dim() == 3 && count > 1 ? t.stride(0) : 0;
    const int64_t ld = std::max((x.cols + 7) & ~int64_t(7), int64_t(8));
    at::Tensor y = t.dim() == 3 ? strided({count, x.rows, x.cols}, {std::max(x.rows * ld, ld), ld, 1}, dtype, t)
                                : strided({x.rows, x.cols}, {ld, 1}, dtype, t);
    at::Tensor work = fresh({gemm_orthogonalize_work_bytes(count, x.rows, x.cols)}, at::kByte, t);
    call("gemm_orthogonalize", [&] {
        return gemm_orthogonalize(type, y_type, count, x.rows, x.cols, x.data(), x.ld, stride, steps, coefficients, eps, y.data_ptr(), ld,
                                  x.rows * ld, work.data_ptr(), stream.handle);
    });
    return wrap(y);
END_BOUND
