"""Routed products on torch CUDA tensors: a router, the experts' products, low-rank adapters.

Tensor-level face of the gemm_moe_*, gemm_grouped_* and gemm_lora_linear entry points of
include/gemm_gb300.h, which states their formulas, masks, limits and alignment rules.  The
functions check types and shapes, create the outputs that are not given, pass addresses, strides
and the current CUDA stream to the library, and raise GemmError on a non-OK status.  Matrices need
unit column stride and may have padded rows; index and weight tensors are contiguous int32 and
fp32.  An expert layer of T tokens, E experts and k experts per token:

    ids, weights, offsets, tokens, where = moe_route(logits, k)      # logits T x E
    h  = grouped_linear(x, w13, offsets, rows=tokens, gated=True)    # w13 E x 2I x H, x T x H
    ys = grouped_linear(h, w2, offsets, out_dtype=torch.float32)     # w2 E x H x I
    y  = moe_combine(ys, where, weights, out_dtype=x.dtype)
"""
from __future__ import annotations

import torch

from ._lib import GEMM_OP_N, GEMM_OP_T, GemmError, load

__all__ = [
    "moe_route", "moe_route_backward", "moe_plan", "moe_dispatch", "moe_combine",
    "moe_combine_backward", "gated_silu_backward", "grouped_linear", "grouped_weight_grad",
    "lora_linear",
]

_F32, _I32 = torch.float32, torch.int32
_TYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_SCORE = {"softmax": 0, "sigmoid": 1}
# the raw handle: building a torch.cuda.Stream for every call costs as much as a launch
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class _Calls:
    """The library's functions, each looked up at its first call."""

    def __getattr__(self, name):
        fn = getattr(load(), name)
        setattr(self, name, fn)
        return fn


_lib = _Calls()


def _raise(status, name):
    raise GemmError(status, name)


def _stream(stream, tensor):
    """The given stream, or the current one of the tensor's device."""
    if stream is None:
        return _raw_stream(tensor.get_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


# The checks' first lines are one condition each: a decoding step's calls are bound by the host.
def _type(dtype, what):
    kind = _TYPE.get(dtype)
    if kind is None:
        raise TypeError(f"{what}: fp32, fp16 or bf16 wanted, got {dtype}")
    return kind


def _refuse(t, what, dims):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: a torch tensor is wanted")
    if not t.is_cuda:
        raise ValueError(f"{what}: must live in CUDA device memory")
    raise ValueError(f"{what}: {dims}-D with unit column stride wanted")


def _matrix(t, what, dims=2):
    """(shape, leading dimension) of a CUDA matrix, or stack of them, with unit column stride."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == dims):
        _refuse(t, what, dims)
    shape, strides = t.shape, t.stride()
    if strides[-1] != 1 and shape[-1] > 1:
        _refuse(t, what, dims)
    ld = strides[-2]
    if shape[-2] <= 1:  # the stride of a single row means nothing
        ld = max(ld, shape[-1], 1)
    return shape, ld


def _same(got, wanted, what):
    if got != wanted:
        raise ValueError(f"{what}: {wanted} wanted, got {got}")


def _same_type(t, dtype, what):
    if t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")


def _array(t, what, dtype, count):
    """Address of a contiguous CUDA array of `count` values."""
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.is_contiguous()
            and t.numel() == count):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: a torch tensor is wanted")
    if not t.is_cuda:
        raise ValueError(f"{what}: must live in CUDA device memory")
    _same_type(t, dtype, what)
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    raise ValueError(f"{what}: {count} values wanted, got {t.numel()}")


def _padded(rows, cols, dtype, device):
    """(matrix, leading dimension): rows start on 16-byte boundaries, multiples of 8 elements."""
    ld = (cols + 7) & ~7
    t = torch.empty((rows, ld), dtype=dtype, device=device)
    return (t, ld) if ld == cols else (t[:, :cols], ld)


def _score(score):
    kind = _SCORE.get(score)
    if kind is None:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    return kind


def moe_route(logits, top_k, *, bias=None, score="softmax", groups=1, groups_kept=1, group_top=1,
              renormalise=True, scale=1.0, stream=None):
    """Experts of every token and the plan of their products: (ids, weights, offsets, tokens, where).

    logits T x E (fp32, fp16 or bf16); ids int32 and weights fp32 are T x top_k; offsets (E + 1),
    tokens and where are the plan (gemm_moe_route).
    """
    (T, E), ld = _matrix(logits, "logits")
    bias = None if bias is None else _array(bias, "bias", _F32, E)
    # one allocation, five views: a view costs half of an allocation and its release
    shape, rows, slots = (T, top_k), (top_k, 1), T * top_k
    space = torch.empty(4 * slots + E + 1, dtype=_I32, device=logits.device)
    weights = space.view(_F32).as_strided(shape, rows, 0)
    ids = space.as_strided(shape, rows, slots)
    where = space.as_strided(shape, rows, 2 * slots)
    tokens = space.as_strided((slots,), (1,), 3 * slots)
    offsets = space.as_strided((E + 1,), (1,), 4 * slots)
    at = space.data_ptr()
    status = _lib.gemm_moe_route(
        _type(logits.dtype, "logits"), T, E, logits.data_ptr(), ld, bias, _score(score), groups,
        groups_kept, group_top, top_k, renormalise, scale, at + 4 * slots, at, at + 16 * slots,
        at + 12 * slots, at + 8 * slots, _stream(stream, logits))
    if status:
        _raise(status, "gemm_moe_route")
    return ids, weights, offsets, tokens, where


def moe_route_backward(dweights, logits, ids, *, score="softmax", renormalise=True, scale=1.0,
                       stream=None):
    """Gradient of moe_route's weights with respect to the logits, ids held fixed."""
    (T, E), ld = _matrix(logits, "logits")
    top_k = ids.shape[1]
    out = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    status = _lib.gemm_moe_route_backward(
        _type(logits.dtype, "logits"), T, E, _array(dweights, "dweights", _F32, T * top_k),
        logits.data_ptr(), ld, _array(ids, "ids", _I32, T * top_k), _score(score), top_k, renormalise,
        scale, out.data_ptr(), E, _stream(stream, logits))
    if status:
        _raise(status, "gemm_moe_route_backward")
    return out


def moe_plan(ids, experts, stream=None):
    """(offsets, tokens, where) of given choices ids (T x k int32; -1: none)."""
    (T, top_k), _ = _matrix(ids, "ids")
    tokens = torch.empty(T * top_k, dtype=_I32, device=ids.device)
    where = torch.empty((T, top_k), dtype=_I32, device=ids.device)
    offsets = torch.empty(experts + 1, dtype=_I32, device=ids.device)
    status = _lib.gemm_moe_plan(T, experts, top_k, _array(ids, "ids", _I32, T * top_k), offsets.data_ptr(),
                                tokens.data_ptr(), where.data_ptr(), _stream(stream, ids))
    if status:
        _raise(status, "gemm_moe_plan")
    return offsets, tokens, where


def moe_dispatch(x, where, weights=None, stream=None):
    """Rows of x (T x H) at the positions of their slots, times the slots' weights if given."""
    (T, H), ld = _matrix(x, "x")
    top_k = where.shape[1]
    slots = T * top_k
    out, ldo = _padded(slots, H, x.dtype, x.device)
    status = _lib.gemm_moe_dispatch(
        _type(x.dtype, "x"), T, H, top_k, x.data_ptr(), ld, _array(where, "where", _I32, slots),
        None if weights is None else _array(weights, "weights", _F32, slots), slots, out.data_ptr(), ldo,
        _stream(stream, x))
    if status:
        _raise(status, "gemm_moe_dispatch")
    return out


def moe_combine(rows, where, weights=None, out_dtype=None, stream=None):
    """y[t] = sum over j of weights[t, j] * rows[where[t, j]] (weights None: 1)."""
    (positions, H), ld = _matrix(rows, "rows")
    T, top_k = where.shape
    slots = T * top_k
    out_dtype = out_dtype or rows.dtype
    y, ldy = _padded(T, H, out_dtype, rows.device)
    status = _lib.gemm_moe_combine(
        _type(rows.dtype, "rows"), _type(out_dtype, "out_dtype"), T, H, top_k, rows.data_ptr(), ld,
        positions, _array(where, "where", _I32, slots),
        None if weights is None else _array(weights, "weights", _F32, slots), y.data_ptr(), ldy,
        _stream(stream, rows))
    if status:
        _raise(status, "gemm_moe_combine")
    return y


def moe_combine_backward(dy, rows, where, weights=None, stream=None):
    """(drows, dweights) of moe_combine: drows of dy's type, dweights fp32 and shaped as where."""
    (T, H), ldd = _matrix(dy, "dy")
    (positions, cols), ldr = _matrix(rows, "rows")
    _same(cols, H, "columns of rows")
    top_k = where.shape[1]
    slots = T * top_k
    drows, ldo = _padded(positions, H, dy.dtype, dy.device)
    dweights = torch.empty((T, top_k), dtype=_F32, device=dy.device)
    status = _lib.gemm_moe_combine_backward(
        _type(dy.dtype, "dy"), _type(rows.dtype, "rows"), T, H, top_k, dy.data_ptr(), ldd, rows.data_ptr(),
        ldr, positions, _array(where, "where", _I32, slots),
        None if weights is None else _array(weights, "weights", _F32, slots), drows.data_ptr(), ldo,
        dweights.data_ptr(), _stream(stream, dy))
    if status:
        _raise(status, "gemm_moe_combine_backward")
    return drows, dweights


def gated_silu_backward(pre, dh, stream=None):
    """dpre = [dgate | dup] of h = silu(gate) * up from pre = [gate | up] and dh."""
    (rows, two), ldp = _matrix(pre, "pre")
    shape, ldh = _matrix(dh, "dh")
    _same(two % 2, 0, "odd columns of pre")
    _same(tuple(shape), (rows, two // 2), "shape of dh")
    out, ldo = _padded(rows, two, pre.dtype, pre.device)
    status = _lib.gemm_gated_silu_backward(
        _type(pre.dtype, "pre"), _type(dh.dtype, "dh"), rows, two // 2, pre.data_ptr(), ldp, dh.data_ptr(),
        ldh, out.data_ptr(), ldo, _stream(stream, pre))
    if status:
        _raise(status, "gemm_gated_silu_backward")
    return out


def grouped_linear(x, w, offsets, *, rows=None, opW="T", gated=False, out_dtype=None, pre=None,
                   stream=None):
    """Y[p] = x[rows[p]] op(w[g]) for the positions p of every group g (offsets: groups + 1 int32).

    w is groups x N x K (opW "T", a linear layer's weight; gated: groups x 2N x K, gate rows first)
    or groups x K x N (opW "N", the layer's input gradient).  rows None: position p reads row p of
    x.  out_dtype: x's type or torch.float32.  pre (gated only): positions x 2N, receives
    [gate | up].
    """
    (x_rows, K), ldx = _matrix(x, "x")
    (groups, w_rows, w_cols), ldw = _matrix(w, "w", 3)
    dtype = x.dtype
    _same_type(w, dtype, "w")
    if opW == "T":
        op, N, inner = GEMM_OP_T, w_rows, w_cols
    elif opW == "N":
        op, N, inner = GEMM_OP_N, w_cols, w_rows
    else:
        raise ValueError(f"opW must be 'T' or 'N', got {opW!r}")
    _same(inner, K, "inner dimension of w")
    if gated:
        _same(N % 2, 0, "odd rows of gated w")
        N //= 2
    y_rows = x_rows if rows is None else rows.numel()
    out_dtype = out_dtype or dtype
    y, ldy = _padded(y_rows, N, out_dtype, x.device)
    at, ldp, work = None, 0, None
    if pre is not None:
        shape, ldp = _matrix(pre, "pre")
        _same_type(pre, dtype, "pre")
        _same(tuple(shape), (y_rows, 2 * N), "shape of pre")
        at = pre.data_ptr()
    if rows is not None:
        rows = _array(rows, "rows", _I32, y_rows)
        if y_rows > 64 * groups:  # space to lay gathered rows out in, where the library would use it
            space = torch.empty(y_rows * ((K + 7) & ~7), dtype=dtype, device=x.device)
            work = space.data_ptr()
    status = _lib.gemm_grouped_linear(
        _type(dtype, "x"), _type(out_dtype, "out_dtype"), groups, _array(offsets, "offsets", _I32, groups + 1),
        op, gated, N, K, x.data_ptr(), ldx, x_rows, rows, w.data_ptr(), ldw, w.stride(0), y.data_ptr(), ldy,
        y_rows, at, ldp, work, _stream(stream, x))
    if status:
        _raise(status, "gemm_grouped_linear")
    return y


def grouped_weight_grad(dy, x, offsets, *, out_dtype=torch.float32, stream=None):
    """dW[g] = sum over the positions p of group g of dy[p]^T x[p]: groups x N x K."""
    (positions, N), ldd = _matrix(dy, "dy")
    (x_rows, K), ldx = _matrix(x, "x")
    _same_type(x, dy.dtype, "x")
    _same(x_rows, positions, "rows of x")
    groups = offsets.numel() - 1
    ld = (K + 7) & ~7
    dw = torch.empty((groups, N, ld), dtype=out_dtype, device=dy.device)
    status = _lib.gemm_grouped_weight_grad(
        _type(dy.dtype, "dy"), _type(out_dtype, "out_dtype"), groups,
        _array(offsets, "offsets", _I32, groups + 1), N, K, dy.data_ptr(), ldd, x.data_ptr(), ldx, positions,
        dw.data_ptr(), ld, N * ld, _stream(stream, dy))
    if status:
        _raise(status, "gemm_grouped_weight_grad")
    return dw if ld == K else dw[:, :, :K]


def lora_linear(x, w, a, b, segments, adapters, *, scales=None, out_dtype=None, stream=None):
    """y[t] = x[t] w^T + scales[i] (x[t] a[i]^T) b[i]^T with i the adapter of token t's request.

    x T x K, w N x K, a adapters x R x K, b adapters x N x R of one 16-bit type; request q owns
    tokens segments[q] .. segments[q + 1] - 1 and uses adapters[q] (int32; -1: none).
    """
    (T, K), ldx = _matrix(x, "x")
    (N, cols), ldw = _matrix(w, "w")
    (count, R, a_cols), lda = _matrix(a, "a", 3)
    shape, ldb = _matrix(b, "b", 3)
    dtype = x.dtype
    if w.dtype != dtype or a.dtype != dtype or b.dtype != dtype:
        for t, what in ((w, "w"), (a, "a"), (b, "b")):
            _same_type(t, dtype, what)
    _same(cols, K, "columns of w")
    _same(a_cols, K, "columns of a")
    _same(tuple(shape), (count, N, R), "shape of b")
    requests = adapters.numel()
    out_dtype = out_dtype or dtype
    y, ldy = _padded(T, N, out_dtype, x.device)
    work = torch.empty(_lib.gemm_lora_work_bytes(T, N, K, requests, R), dtype=torch.uint8, device=x.device)
    status = _lib.gemm_lora_linear(
        _type(dtype, "x"), _type(out_dtype, "out_dtype"), T, N, K, x.data_ptr(), ldx, w.data_ptr(), ldw,
        requests, _array(segments, "segments", _I32, requests + 1), _array(adapters, "adapters", _I32, requests),
        count, R, a.data_ptr(), lda, a.stride(0), b.data_ptr(), ldb, b.stride(0),
        None if scales is None else _array(scales, "scales", _F32, count), y.data_ptr(), ldy, work.data_ptr(),
        _stream(stream, x))
    if status:
        _raise(status, "gemm_lora_linear")
    return y
