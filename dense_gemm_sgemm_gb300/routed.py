"""Routed products on torch CUDA tensors: a router, the experts' products, low-rank adapters.

Tensor-level face of the gemm_moe_*, gemm_grouped_* and gemm_lora_linear entry points of
include/gemm_gb300.h, which states their formulas, masks, limits and alignment rules.  The
functions check types and shapes, create the outputs that are not given, pass addresses, strides
and the current CUDA stream to the library (in the compiled binding csrc/routed_binding.cpp), and
raise TypeError or ValueError on a bad argument, GemmError on a non-OK status.  Matrices need
unit column stride and may have padded rows; index and weight tensors are contiguous int32 and
fp32; all tensors of a call live on one device.  grouped_linear, grouped_weight_grad and lora_linear read
rows in 16-byte pieces: base addresses of 16 bytes and row strides of a multiple of 8 elements (a single
row aside), so a contiguous matrix whose rows are not a multiple of 8 long, a weight too, is padded by the
caller; what these functions return is.  Output rows of positions in no group are left as they were
allocated.  An expert layer of T tokens, E experts and k experts per token:

    ids, weights, offsets, tokens, where = moe_route(logits, k)      # logits T x E
    h  = grouped_linear(x, w13, offsets, rows=tokens, gated=True)    # w13 E x 2I x H, x T x H
    ys = grouped_linear(h, w2, offsets, out_dtype=torch.float32)     # w2 E x H x I
    y  = moe_combine(ys, where, weights, out_dtype=x.dtype)
"""
from __future__ import annotations

import importlib.util
import os

import torch

from . import build
from ._lib import GEMM_OP_N, GEMM_OP_T, GemmError, load

__all__ = [
    "moe_route", "moe_route_backward", "moe_plan", "moe_dispatch", "moe_combine",
    "moe_combine_backward", "gated_silu_backward", "grouped_linear", "grouped_weight_grad",
    "lora_linear",
]


def _load_binding():
    load()  # the library first: without it the error is its own
    if not os.path.exists(build.BINDING_PATH):
        reason = build.binding_error()
        raise ImportError(f"{build.BINDING_PATH} is missing: build it with `python -m dense_gemm_sgemm_gb300.build`"
                          + (f" (the last build made none: {reason})" if reason else ""))
    if build.built_for() != build.torch_abi():
        raise ImportError(f"{build.BINDING_PATH} was built for [{build.built_for() or 'an unknown torch'}], this is "
                          f"[{build.torch_abi()}]: build it again with `python -m dense_gemm_sgemm_gb300.build`")
    spec = importlib.util.spec_from_file_location("_routed", build.BINDING_PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.set_error(GemmError)
    return module


_routed = _load_binding()
_SCORES = {"softmax": 0, "sigmoid": 1}
_OPS = {"N": GEMM_OP_N, "T": GEMM_OP_T}


def _one_of(table, key, what):
    if key not in table:
        raise ValueError(f"{what} must be one of {', '.join(map(repr, table))}, got {key!r}")
    return table[key]


def moe_route(logits, top_k, *, bias=None, score="softmax", groups=1, groups_kept=1, group_top=1,
              renormalise=True, scale=1.0, stream=None):
    """Experts of every token and the plan of their products: (ids, weights, offsets, tokens, where).

    logits T x E (fp32, fp16 or bf16); ids int32 and weights fp32 are T x top_k; offsets (E + 1),
    tokens and where are the plan (gemm_moe_route).
    """
    return _routed.moe_route(logits, top_k, bias, _one_of(_SCORES, score, "score"), groups, groups_kept,
                             group_top, renormalise, scale, stream)


def moe_route_backward(dweights, logits, ids, *, score="softmax", renormalise=True, scale=1.0,
                       stream=None):
    """Gradient of moe_route's weights with respect to the logits, ids held fixed."""
    return _routed.moe_route_backward(dweights, logits, ids, _one_of(_SCORES, score, "score"), renormalise,
                                      scale, stream)


def moe_plan(ids, experts, stream=None):
    """(offsets, tokens, where) of given choices ids (T x k int32; -1: none)."""
    return _routed.moe_plan(ids, experts, stream)


def moe_dispatch(x, where, weights=None, stream=None):
    """Rows of x (T x H) at the positions of their slots, times the slots' weights if given."""
    return _routed.moe_dispatch(x, where, weights, stream)


def moe_combine(rows, where, weights=None, out_dtype=None, stream=None):
    """y[t] = sum over j of weights[t, j] * rows[where[t, j]] (weights None: 1)."""
    return _routed.moe_combine(rows, where, weights, out_dtype, stream)


def moe_combine_backward(dy, rows, where, weights=None, stream=None):
    """(drows, dweights) of moe_combine: drows of dy's type, dweights fp32 and shaped as where."""
    return _routed.moe_combine_backward(dy, rows, where, weights, stream)


def gated_silu_backward(pre, dh, stream=None):
    """dpre = [dgate | dup] of h = silu(gate) * up from pre = [gate | up] and dh."""
    return _routed.gated_silu_backward(pre, dh, stream)


def grouped_linear(x, w, offsets, *, rows=None, opW="T", gated=False, out_dtype=None, pre=None,
                   stream=None):
    """Y[p] = x[rows[p]] op(w[g]) for the positions p of every group g (offsets: groups + 1 int32).

    w is groups x N x K (opW "T", a linear layer's weight; gated: groups x 2N x K, gate rows first)
    or groups x K x N (opW "N", the layer's input gradient).  rows None: position p reads row p of
    x.  out_dtype: x's type or torch.float32.  pre (gated only): positions x 2N, receives
    [gate | up].
    """
    return _routed.grouped_linear(x, w, offsets, rows, _one_of(_OPS, opW, "opW"), gated, out_dtype, pre,
                                  stream)


def grouped_weight_grad(dy, x, offsets, *, out_dtype=torch.float32, stream=None):
    """dW[g] = sum over the positions p of group g of dy[p]^T x[p]: groups x N x K."""
    return _routed.grouped_weight_grad(dy, x, offsets, out_dtype, stream)


def lora_linear(x, w, a, b, segments, adapters, *, scales=None, out_dtype=None, stream=None):
    """y[t] = x[t] w^T + scales[i] (x[t] a[i]^T) b[i]^T with i the adapter of token t's request.

    x T x K, w N x K, a adapters x R x K, b adapters x N x R of one 16-bit type; request q owns
    tokens segments[q] .. segments[q + 1] - 1 and uses adapters[q] (int32; -1: none).
    """
    return _routed.lora_linear(x, w, a, b, segments, adapters, scales, out_dtype, stream)
