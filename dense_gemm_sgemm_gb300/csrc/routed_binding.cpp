// Python binding of the routed products (argument checks, outputs, the C call; see routed.py), and through
// training_binding.h of the block-scaled products and the orthogonalised update.
//
// A decoding step makes several of these calls, each a few microseconds of GPU time.  Checked and
// marshalled in Python one took 11 to 24 us of a Grace core, so the tensors are read here: about 5 us.
// Nothing is computed in this file; every function ends in one call of include/gemm_gb300.h.
#include <ATen/Functions.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <Python.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <optional>

#include "../../include/gemm_gb300.h"

namespace {

PyObject *g_error = nullptr;  // GemmError

// The device of a call's operands: its first tensor's, on whose stream the kernels run.  They read the
// others by their addresses, so a tensor of another device is refused before anything is launched.
struct Device {
    std::optional<c10::Device> of;
    void agree(c10::Device d, const char *what)
    {
        if (!of) of = d;
        TORCH_CHECK_VALUE(d == *of, what, ": on ", d, ", the call's first tensor on ", *of);
    }
};

const at::Tensor &tensor(Device &device, PyObject *o, const char *what)
{
    TORCH_CHECK_TYPE(THPVariable_Check(o), what, ": a torch tensor is wanted");
    const at::Tensor &t = THPVariable_Unpack(o);
    TORCH_CHECK_VALUE(t.is_cuda(), what, ": must live in CUDA device memory");
    device.agree(t.device(), what);
    return t;
}

// A matrix with unit column stride.  The stride of a single row means nothing: any whole number of 16-byte
// pieces that holds the row, so that a row of odd length is not refused for it.
struct Matrix {
    const at::Tensor &t;
    int64_t rows, cols, ld;
    void *data() const { return t.data_ptr(); }
};
Matrix matrix(Device &device, PyObject *o, const char *what, int dims = 2)
{
    const at::Tensor &t = tensor(device, o, what);
    TORCH_CHECK_VALUE(t.dim() == dims && (t.size(-1) <= 1 || t.stride(-1) == 1), what, ": ", dims,
                      "-D with unit column stride wanted");
    const int64_t rows = t.size(-2), cols = t.size(-1);
    int64_t ld = t.stride(-2);
    if (rows <= 1) ld = std::max((cols + 7) & ~int64_t(7), int64_t(8));
    return Matrix{t, rows, cols, ld};
}

void same(int64_t got, int64_t wanted, const char *what)
{
    TORCH_CHECK_VALUE(got == wanted, what, ": ", wanted, " wanted, got ", got);
}
void same_type(const at::Tensor &t, at::ScalarType type, const char *what)
{
    TORCH_CHECK_TYPE(t.scalar_type() == type, what, ": expected ", type, ", got ", t.scalar_type());
}

// A contiguous array of `count` values; None: NULL.
void *array(Device &device, PyObject *o, const char *what, at::ScalarType type, int64_t count, bool optional = false)
{
    if (optional && o == Py_None) return nullptr;
    const at::Tensor &t = tensor(device, o, what);
    same_type(t, type, what);
    TORCH_CHECK_VALUE(t.is_contiguous(), what, ": must be contiguous");
    same(t.numel(), count, what);
    return t.data_ptr();
}
int32_t *ints(Device &device, PyObject *o, const char *what, int64_t count, bool optional = false)
{
    return static_cast<int32_t *>(array(device, o, what, at::kInt, count, optional));
}
float *floats(Device &device, PyObject *o, const char *what, int64_t count, bool optional = false)
{
    return static_cast<float *>(array(device, o, what, at::kFloat, count, optional));
}

gemm_type_t type_of(at::ScalarType t, const char *what)
{
    TORCH_CHECK_TYPE(t == at::kFloat || t == at::kHalf || t == at::kBFloat16, what, ": fp32, fp16 or bf16 wanted, got ", t);
    return t == at::kFloat ? GEMM_TYPE_F32 : t == at::kHalf ? GEMM_TYPE_F16 : GEMM_TYPE_BF16;
}
at::ScalarType dtype_of(PyObject *o, at::ScalarType none)
{
    if (o == Py_None) return none;
    TORCH_CHECK_TYPE(THPDtype_Check(o), "out_dtype: a torch dtype is wanted");
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
int small(PyObject *o)
{
    const int64_t v = integer(o);
    TORCH_CHECK_VALUE(v >= INT_MIN && v <= INT_MAX, "integer out of range: ", v);
    return int(v);
}
float real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return float(v);
}
bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}
// The tensor's device and the given stream, or the device's current one, made current for the call:
// what the call allocates -- its outputs and the space that it releases on return -- belongs to the
// stream that its kernels run on.
struct Stream {
    c10::cuda::CUDAGuard device;
    std::optional<c10::cuda::CUDAStreamGuard> current;
    void *handle;
    Stream(PyObject *o, const at::Tensor &t) : device(t.device())
    {
        if (o == Py_None) {
            handle = c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
            return;
        }
        if (PyLong_Check(o)) {
            handle = reinterpret_cast<void *>(uintptr_t(integer(o)));
        } else {
            PyObject *attr = PyObject_GetAttrString(o, "cuda_stream");
            if (attr == nullptr) throw python_error();
            const pybind11::object owned = pybind11::reinterpret_steal<pybind11::object>(attr);
            handle = reinterpret_cast<void *>(uintptr_t(integer(attr)));
        }
        current.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), t.get_device()));
    }
};

// New memory from torch's allocator (without the dispatcher's way to the same function).
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor &like)
{
    return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}
// Rows on 16-byte boundaries: the leading dimension a multiple of 8 elements.
struct Padded {
    at::Tensor t;
    int64_t ld;
};
Padded padded(int64_t rows, int64_t cols, at::ScalarType type, const at::Tensor &like)
{
    const int64_t ld = (cols + 7) & ~int64_t(7);
    at::Tensor t = fresh({rows, ld}, type, like);
    return Padded{ld == cols ? t : t.narrow(1, 0, cols), ld};
}

// Runs a library call without the interpreter lock; raises GemmError on a status.
template <class F> void call(const char *name, F f)
{
    gemm_status_t status;
    {
        pybind11::gil_scoped_release release;
        status = f();
    }
    if (status == GEMM_OK) return;
    if (PyObject *e = PyObject_CallFunction(g_error, "is", int(status), name)) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }
template <class... T> PyObject *tuple(const T &...t)
{
    const at::Tensor all[] = {t...};
    PyObject *out = PyTuple_New(sizeof...(t));
    if (out == nullptr) throw python_error();
    for (size_t i = 0; i < sizeof...(t); ++i) PyTuple_SET_ITEM(out, i, wrap(all[i]));
    return out;
}

void count_args(Py_ssize_t n, Py_ssize_t wanted)
{
    TORCH_CHECK_TYPE(n == wanted, wanted, " arguments wanted, got ", n);
}

#define BOUND(name, n)                                                              \
    PyObject *name(PyObject *, PyObject *const *a, Py_ssize_t nargs)                \
    {                                                                               \
        HANDLE_TH_ERRORS                                                            \
        count_args(nargs, n);                                                       \
        Device device;
#define END_BOUND          \
    END_HANDLE_TH_ERRORS   \
    }

// logits, top_k, bias, score, groups, groups_kept, group_top, renormalise, scale, stream
BOUND(moe_route, 10)
    const Matrix x = matrix(device, a[0], "logits");
    const Stream stream(a[9], x.t);
    const int64_t T = x.rows, E = x.cols, k = small(a[1]);
    TORCH_CHECK_VALUE(k >= 1 && k <= 1024, "top_k: ", k);
    const gemm_type_t type = type_of(x.t.scalar_type(), "logits");
    const float *bias = floats(device, a[2], "bias", E, true);
    at::Tensor ids = fresh({T, k}, at::kInt, x.t), weights = fresh({T, k}, at::kFloat, x.t);
    at::Tensor offsets = fresh({E + 1}, at::kInt, x.t), tokens = fresh({T * k}, at::kInt, x.t), where = fresh({T, k}, at::kInt, x.t);
    const auto score = static_cast<gemm_score_t>(small(a[3]));
    const int groups = small(a[4]), kept = small(a[5]), top = small(a[6]);
    const bool renormalise = truth(a[7]);
    const float scale = real(a[8]);
    call("gemm_moe_route", [&] {
        return gemm_moe_route(type, T, E, x.data(), x.ld, bias, score, groups, kept, top, int(k), renormalise, scale,
                              ids.data_ptr<int32_t>(), weights.data_ptr<float>(), offsets.data_ptr<int32_t>(),
                              tokens.data_ptr<int32_t>(), where.data_ptr<int32_t>(), stream.handle);
    });
    return tuple(ids, weights, offsets, tokens, where);
END_BOUND

// dweights, logits, ids, score, renormalise, scale, stream
BOUND(moe_route_backward, 7)
    const Matrix x = matrix(device, a[1], "logits"), id = matrix(device, a[2], "ids");
    const Stream stream(a[6], x.t);
    const int64_t T = x.rows, E = x.cols, k = id.cols;
    const gemm_type_t type = type_of(x.t.scalar_type(), "logits");
    const float *dw = floats(device, a[0], "dweights", T * k);
    const int32_t *ids = ints(device, a[2], "ids", T * k);
    at::Tensor out = fresh({T, E}, x.t.scalar_type(), x.t);
    const auto score = static_cast<gemm_score_t>(small(a[3]));
    const bool renormalise = truth(a[4]);
    const float scale = real(a[5]);
    call("gemm_moe_route_backward", [&] {
        return gemm_moe_route_backward(type, T, E, dw, x.data(), x.ld, ids, score, int(k), renormalise, scale, out.data_ptr(), E,
                                       stream.handle);
    });
    return wrap(out);
END_BOUND

// ids, experts, stream
BOUND(moe_plan, 3)
    const Matrix id = matrix(device, a[0], "ids");
    const Stream stream(a[2], id.t);
    const int64_t T = id.rows, k = id.cols, E = integer(a[1]);
    TORCH_CHECK_VALUE(E >= 1 && E <= 1024, "experts: ", E);
    const int32_t *ids = ints(device, a[0], "ids", T * k);
    at::Tensor offsets = fresh({E + 1}, at::kInt, id.t), tokens = fresh({T * k}, at::kInt, id.t), where = fresh({T, k}, at::kInt, id.t);
    call("gemm_moe_plan", [&] {
        return gemm_moe_plan(T, E, int(k), ids, offsets.data_ptr<int32_t>(), tokens.data_ptr<int32_t>(),
                             where.data_ptr<int32_t>(), stream.handle);
    });
    return tuple(offsets, tokens, where);
END_BOUND

// x, where, weights, stream
BOUND(moe_dispatch, 4)
    const Matrix x = matrix(device, a[0], "x"), slot = matrix(device, a[1], "where");
    const Stream stream(a[3], x.t);
    const int64_t T = x.rows, H = x.cols, k = slot.cols, slots = T * k;
    const gemm_type_t type = type_of(x.t.scalar_type(), "x");
    const int32_t *where = ints(device, a[1], "where", slots);
    const float *weights = floats(device, a[2], "weights", slots, true);
    Padded out = padded(slots, H, x.t.scalar_type(), x.t);
    call("gemm_moe_dispatch", [&] {
        return gemm_moe_dispatch(type, T, H, int(k), x.data(), x.ld, where, weights, slots, out.t.data_ptr(), out.ld, stream.handle);
    });
    return wrap(out.t);
END_BOUND

// rows, where, weights, out_dtype, stream
BOUND(moe_combine, 5)
    const Matrix r = matrix(device, a[0], "rows"), slot = matrix(device, a[1], "where");
    const Stream stream(a[4], r.t);
    const int64_t T = slot.rows, k = slot.cols, slots = T * k;
    const gemm_type_t type = type_of(r.t.scalar_type(), "rows");
    const int32_t *where = ints(device, a[1], "where", slots);
    const float *weights = floats(device, a[2], "weights", slots, true);
    const at::ScalarType dtype = dtype_of(a[3], r.t.scalar_type());
    const gemm_type_t y_type = type_of(dtype, "out_dtype");
    Padded y = padded(T, r.cols, dtype, r.t);
    call("gemm_moe_combine", [&] {
        return gemm_moe_combine(type, y_type, T, r.cols, int(k), r.data(), r.ld, r.rows, where, weights, y.t.data_ptr(), y.ld,
                                stream.handle);
    });
    return wrap(y.t);
END_BOUND

// dy, rows, where, weights, stream
BOUND(moe_combine_backward, 5)
    const Matrix dy = matrix(device, a[0], "dy"), r = matrix(device, a[1], "rows"), slot = matrix(device, a[2], "where");
    const Stream stream(a[4], dy.t);
    const int64_t T = dy.rows, H = dy.cols, k = slot.cols, slots = T * k;
    same(r.cols, H, "columns of rows");
    const gemm_type_t type = type_of(dy.t.scalar_type(), "dy"), rows_type = type_of(r.t.scalar_type(), "rows");
    const int32_t *where = ints(device, a[2], "where", slots);
    const float *weights = floats(device, a[3], "weights", slots, true);
    Padded drows = padded(r.rows, H, dy.t.scalar_type(), dy.t);
    at::Tensor dweights = fresh({T, k}, at::kFloat, dy.t);
    call("gemm_moe_combine_backward", [&] {
        return gemm_moe_combine_backward(type, rows_type, T, H, int(k), dy.data(), dy.ld, r.data(), r.ld, r.rows, where, weights,
                                         drows.t.data_ptr(), drows.ld, dweights.data_ptr<float>(), stream.handle);
    });
    return tuple(drows.t, dweights);
END_BOUND

// pre, dh, stream
BOUND(gated_silu_backward, 3)
    const Matrix pre = matrix(device, a[0], "pre"), dh = matrix(device, a[1], "dh");
    const Stream stream(a[2], pre.t);
    same(pre.cols % 2, 0, "odd columns of pre");
    same(dh.rows, pre.rows, "rows of dh");
    same(dh.cols, pre.cols / 2, "columns of dh");
    const gemm_type_t type = type_of(pre.t.scalar_type(), "pre"), dh_type = type_of(dh.t.scalar_type(), "dh");
    Padded out = padded(pre.rows, pre.cols, pre.t.scalar_type(), pre.t);
    call("gemm_gated_silu_backward", [&] {
        return gemm_gated_silu_backward(type, dh_type, pre.rows, dh.cols, pre.data(), pre.ld, dh.data(), dh.ld, out.t.data_ptr(),
                                        out.ld, stream.handle);
    });
    return wrap(out.t);
END_BOUND

// x, w, offsets, rows, op, gated, out_dtype, pre, stream
BOUND(grouped_linear, 9)
    const Matrix x = matrix(device, a[0], "x"), w = matrix(device, a[1], "w", 3);
    const Stream stream(a[8], x.t);
    const at::ScalarType in = x.t.scalar_type(), dtype = dtype_of(a[6], in);
    same_type(w.t, in, "w");
    const gemm_type_t type = type_of(in, "x"), y_type = type_of(dtype, "out_dtype");
    const auto op = static_cast<gemm_op_t>(small(a[4]));
    const bool gated = truth(a[5]);
    const int64_t K = x.cols, groups = w.t.size(0);
    same(op == GEMM_OP_T ? w.cols : w.rows, K, "inner dimension of w");
    int64_t N = op == GEMM_OP_T ? w.rows : w.cols;
    if (gated) {
        same(N % 2, 0, "odd rows of gated w");
        N /= 2;
    }
    const int32_t *offsets = ints(device, a[2], "offsets", groups + 1), *rows = nullptr;
    int64_t y_rows = x.rows;
    if (a[3] != Py_None) {
        y_rows = tensor(device, a[3], "rows").numel();
        rows = ints(device, a[3], "rows", y_rows);
    }
    Padded y = padded(y_rows, N, dtype, x.t);
    void *pre = nullptr;
    int64_t ldp = 0;
    if (a[7] != Py_None) {
        const Matrix m = matrix(device, a[7], "pre");
        same_type(m.t, in, "pre");
        same(m.rows, y_rows, "rows of pre");
        same(m.cols, 2 * N, "columns of pre");
        pre = m.data();
        ldp = m.ld;
    }
    at::Tensor work;  // space to lay gathered rows out in, where the library would use it
    if (rows != nullptr && y_rows > 64 * groups) work = fresh({y_rows * ((K + 63) & ~int64_t(63))}, in, x.t);
    call("gemm_grouped_linear", [&] {
        return gemm_grouped_linear(type, y_type, groups, offsets, op, gated, N, K, x.data(), x.ld, x.rows, rows, w.data(), w.ld,
                                   w.t.stride(0), y.t.data_ptr(), y.ld, y_rows, pre, ldp,
                                   work.defined() ? work.data_ptr() : nullptr, stream.handle);
    });
    return wrap(y.t);
END_BOUND

// dy, x, offsets, out_dtype, stream
BOUND(grouped_weight_grad, 5)
    const Matrix dy = matrix(device, a[0], "dy"), x = matrix(device, a[1], "x");
    const Stream stream(a[4], dy.t);
    const at::ScalarType in = dy.t.scalar_type(), dtype = dtype_of(a[3], at::kFloat);
    same_type(x.t, in, "x");
    same(x.rows, dy.rows, "rows of x");
    const gemm_type_t type = type_of(in, "dy"), dw_type = type_of(dtype, "out_dtype");
    const int64_t groups = tensor(device, a[2], "offsets").numel() - 1, N = dy.cols, K = x.cols, ld = (K + 7) & ~int64_t(7);
    TORCH_CHECK_VALUE(groups >= 0, "offsets: one value at least is wanted");
    const int32_t *offsets = ints(device, a[2], "offsets", groups + 1);
    at::Tensor dw = fresh({groups, N, ld}, dtype, dy.t);
    call("gemm_grouped_weight_grad", [&] {
        return gemm_grouped_weight_grad(type, dw_type, groups, offsets, N, K, dy.data(), dy.ld, x.data(), x.ld, dy.rows,
                                        dw.data_ptr(), ld, N * ld, stream.handle);
    });
    return wrap(ld == K ? dw : dw.narrow(2, 0, K));
END_BOUND

// x, w, a, b, segments, adapters, scales, out_dtype, stream
BOUND(lora_linear, 9)
    const Matrix x = matrix(device, a[0], "x"), w = matrix(device, a[1], "w"), A = matrix(device, a[2], "a", 3), B = matrix(device, a[3], "b", 3);
    const Stream stream(a[8], x.t);
    const at::ScalarType in = x.t.scalar_type(), dtype = dtype_of(a[7], in);
    same_type(w.t, in, "w");
    same_type(A.t, in, "a");
    same_type(B.t, in, "b");
    const gemm_type_t type = type_of(in, "x"), y_type = type_of(dtype, "out_dtype");
    const int64_t T = x.rows, K = x.cols, N = w.rows, R = A.rows, count = A.t.size(0);
    same(w.cols, K, "columns of w");
    same(A.cols, K, "columns of a");
    same(B.t.size(0), count, "adapters of b");
    same(B.rows, N, "rows of b");
    same(B.cols, R, "columns of b");
    const int64_t requests = tensor(device, a[5], "adapters").numel();
    const int32_t *segments = ints(device, a[4], "segments", requests + 1), *adapters = ints(device, a[5], "adapters", requests);
    const float *scales = floats(device, a[6], "scales", count, true);
    Padded y = padded(T, N, dtype, x.t);
    at::Tensor work = fresh({gemm_lora_work_bytes(T, N, K, requests, R)}, at::kByte, x.t);
    call("gemm_lora_linear", [&] {
        return gemm_lora_linear(type, y_type, T, N, K, x.data(), x.ld, w.data(), w.ld, requests, segments, adapters, count, R,
                                A.data(), A.ld, A.t.stride(0), B.data(), B.ld, B.t.stride(0), scales, y.t.data_ptr(), y.ld,
                                work.data_ptr(), stream.handle);
    });
    return wrap(y.t);
END_BOUND

#include "training_binding.h"

// The comparison alone, of two torch devices: first, other.
BOUND(same_device, 2)
    for (int i = 0; i < 2; ++i) {
        TORCH_CHECK_TYPE(THPDevice_Check(a[i]), "a torch device is wanted");
        device.agree(reinterpret_cast<THPDevice *>(a[i])->device, "other");
    }
    Py_RETURN_NONE;
END_BOUND

PyObject *set_error(PyObject *, PyObject *cls)
{
    Py_INCREF(cls);
    Py_XDECREF(g_error);
    g_error = cls;
    Py_RETURN_NONE;
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(moe_route), ENTRY(moe_route_backward), ENTRY(moe_plan), ENTRY(moe_dispatch), ENTRY(moe_combine),
                         ENTRY(moe_combine_backward), ENTRY(gated_silu_backward), ENTRY(grouped_linear),
                         ENTRY(grouped_weight_grad), ENTRY(lora_linear), ENTRY(quantize_blocks), ENTRY(quantize_both),
                         ENTRY(dequantize_blocks), ENTRY(scaled_matmul), ENTRY(orthogonalize), ENTRY(same_device), {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_routed", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__routed(void) { return PyModule_Create(&module); }
