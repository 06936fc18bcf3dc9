"""The router, its plan and its gradient against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import dense_gemm_sgemm_gb300 as g
from tests import routed_reference as ref

pytestmark = pytest.mark.gpu

INF = math.inf


def _logits(T, E, dtype=torch.float32, seed=0, grid=8.0):
    # multiples of 1 / grid: many exact ties, no near ones
    gen = torch.Generator().manual_seed(seed)
    return (torch.randint(-40, 41, (T, E), generator=gen) / grid).to(dtype)


def _check_route(logits, top_k, **kw):
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    ids, w, offsets, tokens, where = g.moe_route(logits.cuda(), top_k, **dev)
    rid, rw = ref.route(logits, top_k, **kw)
    assert torch.equal(ids.cpu().long(), rid)
    # scores: exp and a sum of E terms in fp32, the division and the sum of the chosen
    ref.assert_within(w, rw, 64 * 2.0 ** -24 * (rw.abs() + 1e-30), "weights")
    E = logits.shape[1]
    ro, rt, rp = ref.plan(rid, E)
    assert torch.equal(offsets.cpu().long(), ro)
    assert torch.equal(where.cpu().long(), rp)
    assert torch.equal(tokens.cpu().long()[:rt.numel()], rt)
    return ids, w


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (3, 33, 5), (40, 64, 8), (65, 127, 32), (33, 256, 8),
                                   (20, 300, 6), (9, 513, 32), (7, 1024, 17)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sizes(T, E, k, score):
    _check_route(_logits(T, E, seed=T + E), k, score=score, renormalise=bool(T % 2), scale=1.5)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_16_bit_logits(dtype):
    _check_route(_logits(50, 96, dtype, seed=3), 6, score="sigmoid")


@pytest.mark.parametrize("T", [511, 512, 513, 2100])
def test_one_launch_and_two(T):
    # up to 512 tokens one launch routes and plans
    x = _logits(T, 40, seed=T)
    before = g.gemm_kernel_launches()
    _check_route(x, 4)
    assert g.gemm_kernel_launches() - before == (1 if T <= 512 else 2)


@pytest.mark.parametrize("groups,kept,top", [(2, 1, 1), (4, 2, 2), (8, 8, 2), (32, 5, 1), (16, 3, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [True, False])
def test_groups(groups, kept, top, score, with_bias):
    E = 160
    bias = (torch.randint(-20, 21, (E,), generator=torch.Generator().manual_seed(5)) * 0.013).float()
    k = min(6, E // groups * kept)
    _check_route(_logits(30, E, seed=groups, grid=7.0), k, bias=bias if with_bias else None, score=score,
                 groups=groups, groups_kept=kept, group_top=top, scale=2.5)


def test_masks():
    low = torch.finfo(torch.float32).min
    x = _logits(12, 16, seed=1)
    x[0] = -INF                      # nothing to choose
    x[1] = INF
    x[2] = low
    x[3, 3:] = -INF                  # fewer than k
    x[4, ::2] = math.nan
    x[5] = math.nan
    x[6, 5] = INF
    x[7, :8] = low
    x[8] = 0.0
    x[8, 3] = -0.0                   # equal to +0
    x[9, :15] = -INF
    for score in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            ids, w = _check_route(x, 5, score=score, renormalise=renormalise)
            assert (ids[0] == -1).all() and (w[0] == 0).all() and (ids[5] == -1).all()
            assert torch.isfinite(w).all()
            _check_route(x, 4, score=score, groups=4, groups_kept=2, group_top=2, renormalise=renormalise)
    bias = torch.zeros(16)
    bias[2], bias[3], bias[4] = -INF, math.nan, INF
    ids, _ = _check_route(x, 5, score="sigmoid", bias=bias)
    assert not ((ids == 2) | (ids == 3)).any() and (ids[8, 0] == 4).all()


def test_strided_logits_and_other_stream():
    x = _logits(77, 24, seed=9)
    wide = torch.full((77, 40), math.nan)
    wide[:, :24] = x
    want = ref.route(x, 3)[0]
    s = torch.cuda.Stream()
    dev = wide.cuda()[:, :24]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        ids = g.moe_route(dev, 3)[0]
    s.synchronize()
    assert torch.equal(ids.cpu().long(), want)


def test_no_tokens():
    ids, w, offsets, tokens, where = g.moe_route(torch.empty(0, 12, device="cuda"), 3)
    assert ids.shape == (0, 3) and (offsets == 0).all() and offsets.numel() == 13


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 7, 3), (700, 1024, 3), (3000, 60, 8), (20000, 256, 8)])
def test_plan_of_given_choices(T, E, k):
    rng = np.random.default_rng(T)
    ids = torch.from_numpy(rng.integers(-1, E, (T, k)).astype(np.int32))
    if E > 4:
        ids[ids == 2] = 3            # an expert without slots
        ids[0, 0] = E + 5            # out of range: none
    offsets, tokens, where = (t.cpu().long() for t in g.moe_plan(ids.cuda(), E))
    flat = ids.reshape(-1).long()
    flat = torch.where((flat >= 0) & (flat < E), flat, E)
    at = torch.sort(flat, stable=True).indices
    n = int((flat < E).sum())
    assert torch.equal(offsets, torch.cat([torch.zeros(1, dtype=torch.long),
                                           torch.bincount(flat, minlength=E + 1)[:E].cumsum(0)]))
    assert torch.equal(tokens[:n], at[:n] // k)
    want = torch.full((T * k,), -1)
    want[at[:n]] = torch.arange(n)
    assert torch.equal(where.reshape(-1), want)


def _weights_of(x, ids, score, renormalise, scale):
    s = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)
    w = torch.gather(s, 1, ids.clamp(min=0)) * (ids >= 0)
    if renormalise:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return w * scale


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 40, 3), (65, 256, 8), (9, 1000, 32)])
def test_gradient(T, E, k, score, renormalise):
    gen = torch.Generator().manual_seed(E)
    x = torch.randn(T, E, generator=gen)
    dw = torch.randn(T, k, generator=gen)
    ids = torch.stack([torch.randperm(E, generator=gen)[:k] for _ in range(T)]).int()
    if E > 1:
        ids[0, k - 1] = -1
    got = g.moe_route_backward(dw.cuda(), x.cuda(), ids.cuda(), score=score, renormalise=renormalise,
                               scale=1.7)
    xd = x.double().requires_grad_(True)
    _weights_of(xd, ids.long(), score, renormalise, 1.7).backward(dw.double())
    # every factor is known to about 40 roundings; the sums run over magnitudes up to max |dw|
    s = torch.sigmoid(xd) if score == "sigmoid" else torch.softmax(xd, 1)
    size = 1.7 * dw.abs().max().double() * s.detach()
    if renormalise:
        size = size / torch.gather(s.detach(), 1, ids.long().clamp(min=0)).sum(1, keepdim=True)
    ref.assert_within(got, xd.grad, 2 * 64 * 2.0 ** -24 * size, "dlogits")
    # and against differences of the weights themselves
    d = torch.randn(T, E, generator=gen).double()
    h = 1e-6
    x64 = x.double()
    diff = ((_weights_of(x64 + h * d, ids.long(), score, renormalise, 1.7)
             - _weights_of(x64 - h * d, ids.long(), score, renormalise, 1.7)) / (2 * h) * dw.double()).sum()
    along = (got.double().cpu() * d).sum()
    # differences lose h^2 and 2^-52 / h of sums of T k terms of size 1.7 / S at most
    room = 1e-6 * T * k * 10 * (E if renormalise else 1)
    assert abs(diff - along) <= room, (diff, along)


def test_gradient_of_masked_rows():
    x = torch.randn(4, 10, generator=torch.Generator().manual_seed(2))
    x[0] = -INF
    x[1, 4] = -INF
    x[2] = torch.finfo(torch.float32).min
    ids = torch.tensor([[-1, -1], [0, 7], [0, 1], [3, -1]], dtype=torch.int32)
    for score in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            got = g.moe_route_backward(torch.ones(4, 2, device="cuda"), x.cuda(), ids.cuda(), score=score,
                                       renormalise=renormalise)
            assert torch.isfinite(got).all()
            assert (got[0] == 0).all() and got[1, 4] == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_gradient_16_bit(dtype):
    gen = torch.Generator().manual_seed(8)
    x = torch.randn(30, 64, generator=gen).to(dtype)
    dw = torch.randn(30, 4, generator=gen)
    ids = torch.topk(x.float(), 4, dim=1).indices.int()
    got = g.moe_route_backward(dw.cuda(), x.cuda(), ids.cuda(), renormalise=False)
    xd = x.double().requires_grad_(True)
    _weights_of(xd, ids.long(), "softmax", False, 1.0).backward(dw.double())
    size = dw.abs().max().double() * torch.softmax(xd, 1).detach()
    ref.assert_within(got, xd.grad, 2 * 64 * 2.0 ** -24 * size, "dlogits")


def test_gradient_of_an_expert_named_twice():
    # given choices may repeat an expert: its gradients add up
    x = torch.randn(3, 12, generator=torch.Generator().manual_seed(4))
    ids = torch.tensor([[5, 5, 5], [2, 7, 2], [-1, 3, 3]], dtype=torch.int32)
    dw = torch.tensor([[1.0, -2.0, 0.5], [0.25, 1.0, 3.0], [9.0, 1.0, 1.0]])
    for score in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            got = g.moe_route_backward(dw.cuda(), x.cuda(), ids.cuda(), score=score, renormalise=renormalise)
            xd = x.double().requires_grad_(True)
            _weights_of(xd, ids.long(), score, renormalise, 1.0).backward(dw.double())
            assert (got.double().cpu() - xd.grad).abs().max() <= 64 * 2.0 ** -24 * 10
