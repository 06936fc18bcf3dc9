"""Block-scaled 8-bit matrices on torch CUDA tensors: quantising, reading back, products.

Tensor-level face of the gemm_quantize_*, gemm_dequantize_blocks and gemm_scaled_matmul entry points of
include/gemm_gb300.h, which states their formulas, limits and alignment rules.  The functions check types
and shapes, create the outputs, pass addresses, strides and the current CUDA stream to the library (in
the compiled binding), and raise TypeError or ValueError on a bad argument, GemmError on a non-OK status.
Matrices need unit column stride; 8-bit ones have rows on 16-byte boundaries (a row stride that is a
multiple of 16), as what these functions return does.  Scales are 2-D fp32 tensors of any strides, one
for every block; their shape tells the block.  All tensors of a call live on one device.  No gradient is
recorded: outside torch.no_grad() a tensor that requires one is refused.  A linear layer y = x w^T, its
weight quantised once, and the gradients of its input and weight:

    wq, ws = quantize_blocks(w, (128, 128))                          # w N x K
    xq, xs, xc, xcs = quantize_both(x)                               # x T x K
    y  = scaled_matmul(xq, xs, wq, ws)
    dq, ds, dc, dcs = quantize_both(dy)                              # dy T x N
    dx = scaled_matmul(dq, ds, wq, ws, opB="N")
    dw = scaled_matmul(dc, dcs, xc, xcs, opA="T", opB="N", out_dtype=torch.float32)
"""
from __future__ import annotations

import torch

from .routed import _OPS, _one_of, _routed

__all__ = ["quantize_blocks", "quantize_both", "dequantize_blocks", "scaled_matmul"]

_BLOCKS = {(1, 128): (1, 128), (128, 1): (128, 1), (128, 128): (128, 128)}


def quantize_blocks(x, block=(1, 128), *, dtype=torch.float8_e4m3fn, stream=None):
    """(q, scales) of x in blocks of 1 x 128, 128 x 1 or 128 x 128 elements.

    x rows x cols (fp32, fp16 or bf16); q of dtype (float8_e4m3fn or float8_e5m2) and x's shape; scales
    fp32, ceil(rows / block[0]) x ceil(cols / block[1]), powers of two.
    """
    rows, cols = _one_of(_BLOCKS, block if type(block) is tuple else tuple(block), "block")
    return _routed.quantize_blocks(x, rows, cols, dtype, stream)


def quantize_both(x, *, dtype=torch.float8_e4m3fn, stream=None):
    """(q, scales, qc, scalesc): x in blocks of 1 x 128 and of 128 x 1, in one pass."""
    return _routed.quantize_both(x, dtype, stream)


def dequantize_blocks(q, scales, *, out_dtype=torch.bfloat16, stream=None):
    """The values q * scales stand for, in out_dtype (float32, float16 or bfloat16)."""
    return _routed.dequantize_blocks(q, scales, out_dtype, stream)


def scaled_matmul(A, A_scales, B, B_scales, *, opA="N", opB="T", out_dtype=torch.bfloat16, stream=None):
    """op(A) op(B) of block-scaled 8-bit matrices, M x N of out_dtype (float32, float16 or bfloat16).

    A is stored M x K (opA "N") or K x M ("T"), B K x N (opB "N") or N x K ("T", a linear layer's
    weight); scales are of the stored matrices, for every 128 elements of K and for every one or 128 of
    M or N.
    """
    return _routed.scaled_matmul(A, A_scales, B, B_scales, _one_of(_OPS, opA, "opA"), _one_of(_OPS, opB, "opB"),
                                 out_dtype, stream)
