"""A linear layer trained with 8-bit products and an orthogonalised update of its weight.

Every step: the weight is quantised in blocks of 128 x 128, the activations along their rows (for the forward
product) and along their columns (for the weight's gradient) in one pass, the gradient of the output likewise;
the three products of forward and backward pass run on the 8-bit values; momentum of the weight's gradient is
orthogonalised and taken from the fp32 master weight.  Then the layer serves single tokens with the weight
quantised once, from a captured graph.

    python examples/scaled_layer.py [--steps 20] [--tokens 512] [--inputs 512] [--outputs 384]

prints the loss as it falls and the serving time, and checks the gradients against those of the quantised values.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_sgemm_gb300 as g  # noqa: E402


class ScaledLinear:
    """y = x w^T in 8 bits; forward keeps what backward needs."""

    def __init__(self, inputs, outputs, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.master = torch.randn(outputs, inputs, generator=gen, device="cuda") * inputs ** -0.5
        self.momentum = torch.zeros_like(self.master)
        self.refresh()

    def refresh(self):
        self.w, self.w_scales = g.quantize_blocks(self.master, (128, 128))

    def forward(self, x, keep=False):
        if not keep:
            q, scales = g.quantize_blocks(x)
            return g.scaled_matmul(q, scales, self.w, self.w_scales, out_dtype=x.dtype)
        q, scales, columns, column_scales = g.quantize_both(x)
        return g.scaled_matmul(q, scales, self.w, self.w_scales, out_dtype=x.dtype), (columns, column_scales)

    def backward(self, dy, kept):
        """(dx, dw): gradients have a wider range than activations, so e5m2."""
        q, scales, columns, column_scales = g.quantize_both(dy, dtype=torch.float8_e5m2)
        dx = g.scaled_matmul(q, scales, self.w, self.w_scales, opB="N", out_dtype=dy.dtype)
        dw = g.scaled_matmul(columns, column_scales, *kept, opA="T", opB="N", out_dtype=torch.float32)
        return dx, dw

    def step(self, dw, rate, decay=0.9):
        self.momentum.mul_(decay).add_(dw)
        self.master.add_(g.orthogonalize(self.momentum), alpha=-rate)
        self.refresh()


def train(layer, x, target, steps, rate):
    """Descends half a token's squared error, averaged over the tokens; the mean square error of every step."""
    losses = []
    for _ in range(steps):
        y, kept = layer.forward(x, keep=True)
        diff = y.float() - target
        losses.append(diff.square().mean())
        _, dw = layer.backward((diff / x.shape[0]).to(x.dtype), kept)
        layer.step(dw, rate)
    return [float(v) for v in losses]


def check(layer, x, dy):
    """Largest error of y, dx and dw against fp64 products of what was quantised, relative to each one's norm."""
    values = lambda *qs: g.dequantize_blocks(*qs, out_dtype=torch.float32).double()  # noqa: E731
    y, kept = layer.forward(x, keep=True)
    dx, dw = layer.backward(dy, kept)
    w = values(layer.w, layer.w_scales)
    rows, columns = values(*g.quantize_blocks(x)), values(*kept)
    drows, dcolumns = (values(*g.quantize_blocks(dy, block, dtype=torch.float8_e5m2)) for block in ((1, 128), (128, 1)))
    pairs = (y, rows @ w.T), (dx, drows @ w), (dw, dcolumns.T @ columns)
    return [float((got.double() - want).norm() / want.norm()) for got, want in pairs]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--inputs", type=int, default=512)
    ap.add_argument("--outputs", type=int, default=384)
    ap.add_argument("--rate", type=float, default=0.02)
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.inputs, generator=gen, device="cuda").bfloat16()
    target = x.float() @ torch.randn(a.inputs, a.outputs, generator=gen, device="cuda") * a.inputs ** -0.5
    layer = ScaledLinear(a.inputs, a.outputs)
    losses = train(layer, x, target, a.steps, a.rate)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")
    errors = check(layer, x, ((layer.forward(x).float() - target) / a.tokens).bfloat16())
    print("errors of y, dx, dw against what was quantised: " + ", ".join(f"{e:.1e}" for e in errors))

    token = torch.randn(1, a.inputs, generator=gen, device="cuda").bfloat16()
    graph = torch.cuda.CUDAGraph()  # a decoding loop replays its step
    with torch.cuda.graph(graph):
        served = layer.forward(token)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    if not torch.equal(served, layer.forward(token)):
        raise RuntimeError("a replayed token differs from a computed one")
    print(f"one token: {10 * start.elapsed_time(end):.1f} us a step")
    if g.gemm_get_device_status() != 0:
        raise RuntimeError("device status error")
    return losses, errors


if __name__ == "__main__":
    main()
