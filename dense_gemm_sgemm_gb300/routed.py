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

_TYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_SCORE = {"softmax": 0, "sigmoid": 1}


_calls = {}


def _run(name, *args):
    call = _calls.get(name)
    if call is None:
        call = _calls[name] = getattr(load(), name)
    status = call(*args)
    if status != 0:
        raise GemmError(status, name)


def _stream(stream, tensor):
    """The given stream, or the current one of the tensor's device (the raw handle: building a
    torch.cuda.Stream costs as much as the launch)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(tensor.get_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _type(t, what):
    try:
        return _TYPE[t.dtype]
    except KeyError:
        raise TypeError(f"{what}: fp32, fp16 or bf16 wanted, got {t.dtype}") from None


def _matrix(t, what, cols=None, rows=None, dtype=None, dims=2):
    """Leading dimension of a CUDA tensor with unit column stride (dims = 3: a stack of them)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: a torch tensor is wanted")
    if not t.is_cuda:
        raise ValueError(f"{what}: must live in CUDA device memory")
    shape, strides = t.shape, t.stride()
    if len(shape) != dims or (shape[-1] > 1 and strides[-1] != 1):
        raise ValueError(f"{what}: {dims}-D with unit column stride wanted")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if cols is not None and shape[-1] != cols:
        raise ValueError(f"{what}: {cols} columns wanted, got {shape[-1]}")
    if rows is not None and shape[-2] != rows:
        raise ValueError(f"{what}: {rows} rows wanted, got {shape[-2]}")
    ld = strides[-2]
    # the stride of a single row means nothing
    return ld if shape[-2] > 1 else max(ld, shape[-1], 1)


def _array(t, what, dtype, count=None):
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: a torch tensor is wanted")
    if not t.is_cuda:
        raise ValueError(f"{what}: must live in CUDA device memory")
    if t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    if count is not None and t.numel() != count:
        raise ValueError(f"{what}: {count} values wanted, got {t.numel()}")
    return t.data_ptr()


def _padded(rows, cols, dtype, device):
    """Matrix whose rows start on 16-byte boundaries (leading dimension a multiple of 8)."""
    ld = (cols + 7) // 8 * 8
    t = torch.empty((rows, ld), dtype=dtype, device=device)
    return t if ld == cols else t[:, :cols]


def moe_route(logits, top_k, *, bias=None, score="softmax", groups=1, groups_kept=1, group_top=1,
              renormalise=True, scale=1.0, stream=None):
    """Experts of every token and the plan of their products: (ids, weights, offsets, tokens, where).

    logits T x E (fp32, fp16 or bf16); ids int32 and weights fp32 are T x top_k; offsets (E + 1),
    tokens and where are the plan (gemm_moe_route).
    """
    ld = _matrix(logits, "logits")
    T, E = logits.shape
    dev = logits.device
    weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    where = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    tokens = torch.empty(T * top_k, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    _run("gemm_moe_route", _type(logits, "logits"), T, E, logits.data_ptr(), ld,
         _array(bias, "bias", torch.float32, E), _score(score), groups, groups_kept, group_top, top_k,
         int(renormalise), scale, ids.data_ptr(), weights.data_ptr(), offsets.data_ptr(),
         tokens.data_ptr(), where.data_ptr(), _stream(stream, logits))
    return ids, weights, offsets, tokens, where


def _score(score):
    try:
        return _SCORE[score]
    except KeyError:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}") from None


def moe_route_backward(dweights, logits, ids, *, score="softmax", renormalise=True, scale=1.0,
                       stream=None):
    """Gradient of moe_route's weights with respect to the logits, ids held fixed."""
    ld = _matrix(logits, "logits")
    T, E = logits.shape
    top_k = ids.shape[1]
    out = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    _run("gemm_moe_route_backward", _type(logits, "logits"), T, E,
         _array(dweights, "dweights", torch.float32, T * top_k), logits.data_ptr(), ld,
         _array(ids, "ids", torch.int32, T * top_k), _score(score), top_k, int(renormalise), scale,
         out.data_ptr(), E, _stream(stream, logits))
    return out


def moe_plan(ids, experts, stream=None):
    """(offsets, tokens, where) of given choices ids (T x k int32; -1: none)."""
    addr = _array(ids, "ids", torch.int32)
    T, top_k = ids.shape
    tokens = torch.empty(T * top_k, dtype=torch.int32, device=ids.device)
    where = torch.empty((T, top_k), dtype=torch.int32, device=ids.device)
    offsets = torch.empty(experts + 1, dtype=torch.int32, device=ids.device)
    _run("gemm_moe_plan", T, experts, top_k, addr, offsets.data_ptr(), tokens.data_ptr(),
         where.data_ptr(), _stream(stream, ids))
    return offsets, tokens, where


def moe_dispatch(x, where, weights=None, stream=None):
    """Rows of x (T x H) at the positions of their slots, times the slots' weights if given."""
    ld = _matrix(x, "x")
    T, H = x.shape
    top_k = where.shape[1]
    out = _padded(T * top_k, H, x.dtype, x.device)
    _run("gemm_moe_dispatch", _type(x, "x"), T, H, top_k, x.data_ptr(), ld,
         _array(where, "where", torch.int32, T * top_k),
         _array(weights, "weights", torch.float32, T * top_k), T * top_k, out.data_ptr(),
         out.stride(0), _stream(stream, x))
    return out


def moe_combine(rows, where, weights=None, out_dtype=None, stream=None):
    """y[t] = sum over j of weights[t, j] * rows[where[t, j]] (weights None: 1)."""
    ld = _matrix(rows, "rows")
    T, top_k = where.shape
    H = rows.shape[1]
    y = _padded(T, H, out_dtype or rows.dtype, rows.device)
    _run("gemm_moe_combine", _type(rows, "rows"), _type(y, "out_dtype"), T, H, top_k, rows.data_ptr(),
         ld, rows.shape[0], _array(where, "where", torch.int32),
         _array(weights, "weights", torch.float32, T * top_k), y.data_ptr(), y.stride(0),
         _stream(stream, rows))
    return y


def moe_combine_backward(dy, rows, where, weights=None, stream=None):
    """(drows, dweights) of moe_combine: drows of dy's type, dweights fp32 and shaped as where."""
    T, H = dy.shape
    ldd, ldr = _matrix(dy, "dy"), _matrix(rows, "rows", cols=H)
    top_k = where.shape[1]
    drows = _padded(rows.shape[0], H, dy.dtype, dy.device)
    dweights = torch.empty((T, top_k), dtype=torch.float32, device=dy.device)
    _run("gemm_moe_combine_backward", _type(dy, "dy"), _type(rows, "rows"), T, H, top_k, dy.data_ptr(),
         ldd, rows.data_ptr(), ldr, rows.shape[0], _array(where, "where", torch.int32, T * top_k),
         _array(weights, "weights", torch.float32, T * top_k), drows.data_ptr(), drows.stride(0),
         dweights.data_ptr(), _stream(stream, dy))
    return drows, dweights


def gated_silu_backward(pre, dh, stream=None):
    """dpre = [dgate | dup] of h = silu(gate) * up from pre = [gate | up] and dh."""
    ldp = _matrix(pre, "pre")
    rows, two = pre.shape
    if two % 2:
        raise ValueError("pre: an even number of columns is wanted")
    ldh = _matrix(dh, "dh", cols=two // 2, rows=rows)
    out = _padded(rows, two, pre.dtype, pre.device)
    _run("gemm_gated_silu_backward", _type(pre, "pre"), _type(dh, "dh"), rows, two // 2, pre.data_ptr(),
         ldp, dh.data_ptr(), ldh, out.data_ptr(), out.stride(0), _stream(stream, pre))
    return out


def grouped_linear(x, w, offsets, *, rows=None, opW="T", gated=False, out_dtype=None, pre=None,
                   stream=None):
    """Y[p] = x[rows[p]] op(w[g]) for the positions p of every group g (offsets: groups + 1 int32).

    w is groups x N x K (opW "T", a linear layer's weight; gated: groups x 2N x K, gate rows first)
    or groups x K x N (opW "N", the layer's input gradient).  rows None: position p reads row p of
    x.  out_dtype: x's type or torch.float32.  pre (gated only): positions x 2N, receives
    [gate | up].
    """
    ldx = _matrix(x, "x")
    x_rows, K = x.shape
    if opW not in ("T", "N"):
        raise ValueError(f"opW must be 'T' or 'N', got {opW!r}")
    ldw = _matrix(w, "w", dtype=x.dtype, dims=3, cols=K if opW == "T" else None,
                  rows=K if opW == "N" else None)
    groups = w.shape[0]
    N = w.shape[1] if opW == "T" else w.shape[2]
    if gated:
        if N % 2:
            raise ValueError("w: gated weights have gate and up rows, an even number")
        N //= 2
    y_rows = x_rows if rows is None else rows.numel()
    y = _padded(y_rows, N, out_dtype or x.dtype, x.device)
    ldp = 0
    if pre is not None:
        ldp = _matrix(pre, "pre", cols=2 * N, rows=y_rows, dtype=x.dtype)
    # space to lay gathered rows out in, where the library would use it
    work = None
    if rows is not None and y_rows > 64 * groups:
        space = torch.empty(y_rows * ((K + 7) // 8 * 8), dtype=x.dtype, device=x.device)
        work = space.data_ptr()
    _run("gemm_grouped_linear", _type(x, "x"), _type(y, "out_dtype"), groups,
         _array(offsets, "offsets", torch.int32, groups + 1), GEMM_OP_T if opW == "T" else GEMM_OP_N,
         int(gated), N, K, x.data_ptr(), ldx, x_rows, _array(rows, "rows", torch.int32), w.data_ptr(),
         ldw, w.stride(0), y.data_ptr(), y.stride(0), y_rows, 0 if pre is None else pre.data_ptr(), ldp,
         work, _stream(stream, x))
    return y


def grouped_weight_grad(dy, x, offsets, *, out_dtype=torch.float32, stream=None):
    """dW[g] = sum over the positions p of group g of dy[p]^T x[p]: groups x N x K."""
    ldd, ldx = _matrix(dy, "dy"), _matrix(x, "x", rows=dy.shape[0], dtype=dy.dtype)
    N, K = dy.shape[1], x.shape[1]
    groups = offsets.numel() - 1
    ld = (K + 7) // 8 * 8
    dw = torch.empty((groups, N, ld), dtype=out_dtype, device=dy.device)
    _run("gemm_grouped_weight_grad", _type(dy, "dy"), _type(dw, "out_dtype"), groups,
         _array(offsets, "offsets", torch.int32), N, K, dy.data_ptr(), ldd, x.data_ptr(), ldx,
         dy.shape[0], dw.data_ptr(), ld, N * ld, _stream(stream, dy))
    return dw if ld == K else dw[:, :, :K]


def lora_linear(x, w, a, b, segments, adapters, *, scales=None, out_dtype=None, stream=None):
    """y[t] = x[t] w^T + scales[i] (x[t] a[i]^T) b[i]^T with i the adapter of token t's request.

    x T x K, w N x K, a adapters x R x K, b adapters x N x R of one 16-bit type; request q owns
    tokens segments[q] .. segments[q + 1] - 1 and uses adapters[q] (int32; -1: none).
    """
    ldx = _matrix(x, "x")
    T, K = x.shape
    dt = x.dtype
    ldw = _matrix(w, "w", cols=K, dtype=dt)
    N = w.shape[0]
    lda = _matrix(a, "a", cols=K, dtype=dt, dims=3)
    count, R = a.shape[0], a.shape[1]
    ldb = _matrix(b, "b", cols=R, rows=N, dtype=dt, dims=3)
    if b.shape[0] != count:
        raise ValueError(f"b: {count} adapters wanted, got {b.shape[0]}")
    requests = adapters.numel()
    y = _padded(T, N, out_dtype or dt, x.device)
    work = torch.empty(load().gemm_lora_work_bytes(T, requests, R), dtype=torch.uint8, device=x.device)
    _run("gemm_lora_linear", _type(x, "x"), _type(y, "out_dtype"), T, N, K, x.data_ptr(), ldx,
         w.data_ptr(), ldw, requests, _array(segments, "segments", torch.int32, requests + 1),
         _array(adapters, "adapters", torch.int32), count, R, a.data_ptr(), lda, a.stride(0),
         b.data_ptr(), ldb, b.stride(0), _array(scales, "scales", torch.float32, count), y.data_ptr(),
         y.stride(0), work.data_ptr(), _stream(stream, x))
    return y
