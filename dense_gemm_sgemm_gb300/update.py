"""The orthogonalised update of a weight on torch CUDA tensors.

Tensor-level face of gemm_orthogonalize of include/gemm_gb300.h, which states its formula, precision and
limits.  The function checks types and shapes, creates the output and the call's work space, passes
addresses, strides and the current CUDA stream to the library (in the compiled binding), and raises
TypeError or ValueError on a bad argument (outside torch.no_grad() a g that requires a gradient is one: none
is recorded), GemmError on a non-OK status.  One step of an optimiser with
momentum m of a weight w (both fp32) and gradient g:

    m.mul_(0.95).add_(g)
    w.add_(orthogonalize(m), alpha=-lr)
"""
from __future__ import annotations

import torch

from .routed import _routed

__all__ = ["orthogonalize"]

_QUINTIC = (3.4445, -4.7750, 2.0315)


def orthogonalize(g, *, steps=5, coefficients=_QUINTIC, eps=1e-7, out_dtype=torch.bfloat16, stream=None):
    """The update of g (rows x cols, or a stack of such matrices; fp32, fp16 or bf16), in out_dtype and g's shape.

    coefficients: (a, b, c) of a X + (b A + c A A) X, A = X X^T, or one such triple for each step.
    out_dtype: bfloat16, float32 or float16, to which the same result is rounded.
    """
    each = tuple(coefficients)
    if each and not isinstance(each[0], (tuple, list)):
        each = (each,) * steps
    if any(len(c) != 3 for c in each):
        raise ValueError("coefficients: three for each step wanted")
    return _routed.orthogonalize(g, steps, tuple(v for c in each for v in c), eps, out_dtype, stream)
