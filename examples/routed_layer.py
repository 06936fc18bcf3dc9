"""A small model block with everything of the routed products in it, trained and then served.

Training: tokens go through a router, the chosen experts' gated products and the weighted sum; the
gradient comes back through all of them, and plain gradient descent steps the router and the experts.
Serving: the same block decodes batches of requests whose shared projection in front of the router
carries a low-rank adapter for each request.  The router's logits come from the library's own GEMM.

    python examples/routed_layer.py [--steps 20] [--tokens 512] [--hidden 256] [--inner 128]

prints the loss as it falls and the serving rate, and checks one decoded batch against torch.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_sgemm_gb300 as g  # noqa: E402


class ExpertLayer:
    """Router and experts; forward keeps what backward needs."""

    def __init__(self, hidden, inner, experts, top_k, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s, std: torch.randn(*s, generator=gen, device="cuda") * std  # noqa: E731
        self.top_k, self.experts, self.dtype = top_k, experts, dtype
        # fp32 master weights, stepped by the optimizer, and the 16-bit copies the products read
        self.master = {"router": rnd(experts, hidden, std=hidden ** -0.5),
                       "w13": rnd(experts, 2 * inner, hidden, std=hidden ** -0.5),
                       "w2": rnd(experts, hidden, inner, std=inner ** -0.5)}
        self.refresh()

    def refresh(self):
        self.w = {name: t.to(self.dtype) for name, t in self.master.items()}

    def forward(self, x, keep=False):
        logits = g.matmul(x, self.w["router"], opB="T")  # fp32 T x experts
        ids, weights, offsets, tokens, where = g.moe_route(logits, self.top_k)
        pre = None
        if keep:
            pre = torch.empty(tokens.numel(), self.w["w13"].shape[1], dtype=self.dtype, device=x.device)
        h = g.grouped_linear(x, self.w["w13"], offsets, rows=tokens, gated=True, pre=pre)
        rows = g.grouped_linear(h, self.w["w2"], offsets, out_dtype=torch.float32)
        y = g.moe_combine(rows, where, weights, out_dtype=self.dtype)
        return (y, (x, logits, ids, weights, offsets, tokens, where, pre, h, rows)) if keep else y

    def backward(self, dy, kept):
        x, logits, ids, weights, offsets, tokens, where, pre, h, rows = kept
        drows, dweights = g.moe_combine_backward(dy, rows, where, weights)
        dw2 = g.grouped_weight_grad(drows, h, offsets)
        dh = g.grouped_linear(drows, self.w["w2"], offsets, opW="N")
        dpre = g.gated_silu_backward(pre, dh)
        dw13 = g.grouped_weight_grad(dpre, g.moe_dispatch(x, where), offsets)
        dxs = g.grouped_linear(dpre, self.w["w13"], offsets, opW="N", out_dtype=torch.float32)
        dx = g.moe_combine(dxs, where, out_dtype=torch.float32)
        dlogits = g.moe_route_backward(dweights, logits, ids).to(self.dtype)
        dx += g.matmul(dlogits, self.w["router"])
        drouter = g.matmul(dlogits, x, opA="T")
        return dx, {"router": drouter, "w13": dw13, "w2": dw2}

    def step(self, grads, rate):
        for name, grad in grads.items():
            self.master[name] -= rate * grad
        self.refresh()


def train(layer, tokens, hidden, steps, rate):
    """Fits the layer to a fixed random target by descending half a token's squared error, averaged over
    the tokens; the mean square error of every step."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, hidden, generator=gen, device="cuda").to(layer.dtype)
    target = torch.randn(tokens, hidden, generator=gen, device="cuda")
    losses = []
    for _ in range(steps):
        y, kept = layer.forward(x, keep=True)
        diff = y.float() - target
        losses.append(diff.square().mean())
        _, grads = layer.backward((diff / tokens).to(layer.dtype), kept)
        layer.step(grads, rate)
    return [float(v) for v in losses]


class Served:
    """The layer behind a shared projection with an adapter of each request."""

    def __init__(self, layer, hidden, adapters, rank, seed=2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s, std: (torch.randn(*s, generator=gen, device="cuda") * std).to(layer.dtype)  # noqa: E731
        self.layer = layer
        self.w = rnd(hidden, hidden, std=hidden ** -0.5)
        self.a = rnd(adapters, rank, hidden, std=hidden ** -0.5)
        self.b = rnd(adapters, hidden, rank, std=rank ** -0.5)

    def decode(self, x, segments, adapters):
        return self.layer.forward(g.lora_linear(x, self.w, self.a, self.b, segments, adapters))


def plain(served, x, segments, adapters):
    """decode() in torch, one request and one token at a time."""
    w, layer = {k: v.float() for k, v in served.layer.w.items()}, served.layer
    z = x.float() @ served.w.float().T
    for q, a in enumerate(adapters.tolist()):
        r = slice(int(segments[q]), int(segments[q + 1]))
        if a >= 0:
            z[r] += x[r].float() @ served.a[a].float().T @ served.b[a].float().T
    z = z.to(layer.dtype).float()
    p = torch.softmax(z @ w["router"].T, dim=1)
    top = torch.topk(p, layer.top_k, dim=1)
    y = torch.zeros_like(z)
    for t in range(z.shape[0]):
        for j, e in enumerate(top.indices[t].tolist()):
            gate, up = (w["w13"][e] @ z[t]).chunk(2)
            y[t] += top.values[t, j] / top.values[t].sum() * (w["w2"][e] @ (torch.nn.functional.silu(gate) * up))
    return y


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=256)
    ap.add_argument("--inner", type=int, default=128)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top-k", type=int, default=2)
    ap.add_argument("--rate", type=float, default=0.1)
    a = ap.parse_args(argv)
    layer = ExpertLayer(a.hidden, a.inner, a.experts, a.top_k)
    losses = train(layer, a.tokens, a.hidden, a.steps, a.rate)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")

    served = Served(layer, a.hidden, adapters=8, rank=8)
    # a decoding batch: 20 requests of one token, two prompts of 9 and 30 tokens, one without adapter
    lengths = [1] * 20 + [9, 30]
    segments = torch.tensor([0] + lengths).cumsum(0).int().cuda()
    adapters = (torch.arange(len(lengths)) % 9 - 1).int().cuda()
    x = torch.randn(sum(lengths), a.hidden, generator=torch.Generator(device="cuda").manual_seed(3),
                    device="cuda").to(layer.dtype)
    y, want = served.decode(x, segments, adapters), plain(served, x, segments, adapters)
    error = float((y.float() - want).norm() / want.norm())
    graph = torch.cuda.CUDAGraph()  # a decoding loop replays its step
    with torch.cuda.graph(graph):
        served.decode(x, segments, adapters)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"decoded {len(lengths)} requests, relative error {error:.1e}, {10 * start.elapsed_time(end):.1f} us a step")
    if g.gemm_get_device_status() != 0:
        raise RuntimeError("device status error")
    return losses, error


if __name__ == "__main__":
    main()
