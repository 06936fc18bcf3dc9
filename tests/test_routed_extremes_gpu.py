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
