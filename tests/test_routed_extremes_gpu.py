"""Routed products at values, strides and hand-overs that ordinary calls seldom meet."""
import pytest
import torch

import dense_gemm_sgemm_gb300 as g
from tests import routed_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_where_the_chosen_scores_are_tiny(score):
    # a balancing bias may choose experts of scores near fp32's smallest normal number: their renormalised
    # weights are ordinary, and so is the gradient, though 1 / (sum of the scores) is not
    gen = torch.Generator().manual_seed(1)
    T, E, k, scale = 50, 40, 4, 2.5
    x = -86.9 + 0.25 * torch.rand(T, E, generator=gen)
    ids = torch.argsort(torch.rand(T, E, generator=gen), dim=1)[:, :k].int()
    if score == "softmax":
        x[:, E - 1] = 0.0
        ids[ids == E - 1] = E // 2
    dw = 100.0 * torch.randn(T, k, generator=gen)
    got = g.moe_route_backward(dw.cuda(), x.cuda(), ids.cuda(), score=score, scale=scale)
    # in 64 bits: dx = scale * p (dw - sum dw p), times 1 - s for a sigmoid; an expert named twice sums
    s = torch.softmax(x.double(), 1) if score == "softmax" else torch.sigmoid(x.double())
    chosen = torch.gather(s, 1, ids.long())
    p = chosen / chosen.sum(1, keepdim=True)
    d = scale * p * (dw.double() - (dw.double() * p).sum(1, keepdim=True))
    size = scale * p * (dw.double().abs() + (dw.double() * p).abs().sum(1, keepdim=True))
    if score == "sigmoid":
        d = d * (1.0 - chosen)
    want = torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, ids.long(), d)
    # the scores' exponentials and sum, then a dozen roundings
    bound = torch.zeros_like(want).scatter_add_(1, ids.long(), 64 * 2.0 ** -24 * size)
    ref.assert_within(got, want, bound)


def test_one_row_has_no_stride():
    # a single row of a row length that is no multiple of 8: nothing is read past it, so it is not refused
    gen = torch.Generator().manual_seed(2)
    K, N = 1003, 37
    x = torch.randn(1, K, generator=gen).half()
    w = torch.zeros(2, N, 1008).half()
    w[..., :K] = torch.randn(2, N, K, generator=gen) * K ** -0.5
    w = w.cuda()[..., :K]
    want, size = x.double() @ w[1].double().cpu().T, x.double().abs() @ w[1].double().cpu().abs().T
    bound = ref.sum_bound(K) * size
    for off in ([0, 0, 1], [0, 0, 90]):
        rows = torch.zeros(off[-1], dtype=torch.int32, device="cuda")
        y = g.grouped_linear(x.cuda(), w, torch.tensor(off, dtype=torch.int32, device="cuda"), rows=rows)
        ref.assert_within(y, want.expand(off[-1], N), bound.expand(off[-1], N))
    none = torch.tensor([-1], dtype=torch.int32, device="cuda")
    a, b = torch.zeros(1, 8, 1008, dtype=torch.float16, device="cuda")[..., :K], torch.zeros(1, N, 8, dtype=torch.float16, device="cuda")
    y = g.lora_linear(x.cuda(), w[1], a, b, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), none)
    ref.assert_within(y, want, bound)
    dy = torch.randn(1, N, generator=gen).half()
    dw = g.grouped_weight_grad(dy.cuda(), x.cuda(), torch.tensor([0, 1], dtype=torch.int32, device="cuda"))
    outer = dy.double().T @ x.double()
    ref.assert_within(dw[0], outer, ref.sum_bound(1) * outer.abs())


@pytest.mark.parametrize("T,requests", [(60, 60), (4096, 5), (700, 90)])
def test_layer_with_adapters_right_behind_what_writes_its_inputs(T, requests):
    # the projection starts before the inner products' kernel has ended, which itself starts while the
    # kernel ahead still runs: that one writes x, the segments or the adapters, many megabytes late
    gen = torch.Generator().manual_seed(T)
    H, k, n, R = 1024, 8, 6, 16
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).half().cuda()  # noqa: E731
    w, a, b = rnd(264, H, std=H ** -0.5), rnd(n, R, H, std=H ** -0.5), rnd(n, 264, R, std=R ** -0.5)
    big = 8192
    rows = [torch.randn(big * k, H, generator=gen).half().cuda() for _ in range(2)]
    where = torch.randperm(big * k, generator=gen).int().reshape(big, k).cuda()
    cuts = [torch.cat([torch.tensor([0]), torch.sort(torch.randint(0, T + 1, (requests - 1,), generator=gen)).values,
                       torch.tensor([T])]).int().cuda() for _ in range(2)]
    who = [torch.randint(-1, n, (requests,), generator=gen).int().cuda() for _ in range(2)]

    def call(i, late):
        # `late`: the operand whose writer is the last kernel ahead
        x = torch.empty(0)
        segments, adapters = torch.zeros_like(cuts[0]), torch.zeros_like(who[0])
        if late != "x":
            x = g.moe_combine(rows[i], where)[-T:]
        segments.copy_(cuts[i])
        adapters.copy_(who[i])
        if late == "x":
            x = g.moe_combine(rows[i], where)[-T:]
        else:
            # a long kernel, then the operand itself
            junk = torch.empty(1 << 28, dtype=torch.uint8, device="cuda").fill_(i)
            if late == "segments":
                segments.zero_()
                segments.add_(cuts[i] + 0 * junk[:1].int())
            else:
                adapters.fill_(-1)
                adapters.copy_(who[i] + 0 * junk[:1].int())
        return g.lora_linear(x, w, a, b, segments, adapters)

    want = []
    for i in range(2):
        x = g.moe_combine(rows[i], where)[-T:].clone()
        torch.cuda.synchronize()
        want.append(g.lora_linear(x, w, a, b, cuts[i], who[i]))
        torch.cuda.synchronize()
    for late in ("x", "segments", "adapters"):
        for i in (0, 1, 0, 1):
            y = call(i, late)
            torch.cuda.synchronize()
            assert torch.equal(y, want[i])
    assert g.gemm_get_device_status() == 0


@pytest.mark.parametrize("T,E,k,H,I", [(5, 8, 2, 256, 128), (700, 16, 4, 512, 256), (4000, 24, 3, 1000, 264)])
def test_chained_calls_read_what_the_call_before_wrote(T, E, k, H, I):
    # each kernel may be on the SMs before the one ahead has ended; two inputs in turn go through the same
    # memory, so that anything read too early is the other input's
    gen = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    w13, w2, wl = rnd(E, 2 * I, H), rnd(E, H, I), rnd(H, H)
    a, b = rnd(6, 8, H), rnd(6, H, 8)
    xs = [rnd(T, H) for _ in range(2)]
    logits = [torch.randn(T, E, generator=gen, device="cuda") for _ in range(2)]
    segments = torch.tensor([0, T // 3, T // 2, T], dtype=torch.int32, device="cuda")
    who = torch.tensor([2, -1, 5], dtype=torch.int32, device="cuda")

    def layer(i):
        ids, wt, off, tokens, where = g.moe_route(logits[i], k)
        pre = torch.empty(T * k, 2 * I, dtype=torch.bfloat16, device="cuda")
        h = g.grouped_linear(xs[i], w13, off, rows=tokens, gated=True, pre=pre)
        ys = g.grouped_linear(h, w2, off, out_dtype=torch.float32)
        y = g.moe_combine(ys, where, wt, out_dtype=torch.bfloat16)
        z = g.lora_linear(y, wl, a, b, segments, who)
        drows, dwt = g.moe_combine_backward(z, ys, where, wt)
        dw2 = g.grouped_weight_grad(drows, h, off)
        dpre = g.gated_silu_backward(pre, g.grouped_linear(drows, w2, off, opW="N"))
        dw13 = g.grouped_weight_grad(dpre, g.moe_dispatch(xs[i], where), off)
        return z, dwt, dw2, dw13, g.moe_route_backward(dwt, logits[i], ids)

    want = []
    for i in range(2):
        want.append([t.clone() for t in layer(i)])
        torch.cuda.synchronize()
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for n in range(12):
        out = layer(n & 1)
        for got, ref_ in zip(out, want[n & 1]):
            wrong += (got != ref_).sum()
        del out
    assert int(wrong) == 0
