"""Routed products where they can go wrong besides their values: expired waits, streams that are not the
current one, offsets past 32 bits, refused arguments on the device's side."""
import math

import pytest
import torch

import dense_gemm_sgemm_gb300 as g
from tests import routed_reference as ref

pytestmark = pytest.mark.gpu

TIMEOUT = 5  # GEMM_ERR_DEVICE_TIMEOUT


def _rand(*shape, dtype=torch.float16, seed=0):
    return torch.randint(-2, 3, shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def _calls():
    """Each tcgen05 form with its exact value (small integers: every sum is exact)."""
    P, N, K = 300, 264, 192
    x, w, wn = _rand(P, K), _rand(2, N, K, seed=1), _rand(2, K, N, seed=2)
    off = torch.tensor([0, 170, P], dtype=torch.int32, device="cuda")
    a, b = _rand(3, 8, K, seed=3), _rand(3, N, 8, seed=4)
    ad = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    halves = (slice(0, 170), slice(170, P))
    f = torch.float32

    def pick(parts):
        return torch.cat(parts)

    yield (lambda: g.grouped_linear(x, w, off, out_dtype=f), pick([x[s].float() @ w[i].float().T for i, s in enumerate(halves)]))
    yield (lambda: g.grouped_linear(x, wn, off, opW="N", out_dtype=f),
           pick([x[s].float() @ wn[i].float() for i, s in enumerate(halves)]))
    yield (lambda: g.grouped_weight_grad(x, x, off), torch.stack([x[s].float().T @ x[s].float() for s in halves]))
    inner = [x[s].float() @ a[i].float().T for s, i in zip(halves, (2, 0))]
    yield (lambda: g.lora_linear(x, w[0], a, b, off, ad, out_dtype=f),
           pick([x[s].float() @ w[0].float().T + t @ b[i].float().T for s, i, t in zip(halves, (2, 0), inner)]))


@pytest.mark.parametrize("which", range(4))
def test_expired_wait_is_reported_and_context_survives(monkeypatch, which):
    call, want = list(_calls())[which]
    assert g.gemm_get_device_status() == 0
    monkeypatch.setenv("GEMM_GB300_TEST_INJECT_STALL", "1")
    call()
    assert g.gemm_get_device_status() == TIMEOUT
    assert g.gemm_get_device_status() == 0
    monkeypatch.delenv("GEMM_GB300_TEST_INJECT_STALL")
    assert torch.equal(call(), want)
    assert g.gemm_get_device_status() == 0


@pytest.mark.parametrize("as_handle", [False, True])
def test_given_stream_keeps_its_memory(as_handle):
    # the call's outputs and its space belong to the given stream: the current stream's next
    # allocations of the same size must not reuse them while the call's kernels still run
    gen = torch.Generator(device="cuda").manual_seed(3)
    E, c, H, I = 4, 600, 512, 256
    x = torch.randn(E * c // 2, H, generator=gen, device="cuda").half()
    w = torch.randn(E, 2 * I, H, generator=gen, device="cuda").half()
    off = (torch.arange(E + 1) * c).int().cuda()
    rows = torch.randint(0, x.shape[0], (E * c,), generator=gen, device="cuda").int()
    want = g.grouped_linear(x, w, off, rows=rows, gated=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        y = g.grouped_linear(x, w, off, rows=rows, gated=True, stream=side.cuda_stream if as_handle else side)
        junk = [torch.full((E * c, H), math.nan, dtype=torch.float16, device="cuda") for _ in range(3)]
        del junk
        side.synchronize()
        assert torch.equal(y, want)


def test_calls_on_two_streams_at_once():
    gen = torch.Generator(device="cuda").manual_seed(5)
    T, E, k, H, I = 700, 16, 4, 256, 128
    w13 = torch.randn(E, 2 * I, H, generator=gen, device="cuda").bfloat16()
    w2 = torch.randn(E, H, I, generator=gen, device="cuda").bfloat16()
    xs = [torch.randn(T, H, generator=gen, device="cuda").bfloat16() for _ in range(2)]
    logits = [torch.randn(T, E, generator=gen, device="cuda") for _ in range(2)]

    def layer(i):
        ids, wt, off, tokens, where = g.moe_route(logits[i], k)
        h = g.grouped_linear(xs[i], w13, off, rows=tokens, gated=True)
        return g.moe_combine(g.grouped_linear(h, w2, off, out_dtype=torch.float32), where, wt)

    want = [layer(0), layer(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        got = []
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got.append(layer(i))
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(got[i], want[i])


def test_weights_past_32_bits():
    # the last group's weights start beyond 2^31 elements; only it has rows, few and many
    E, N, K = 270, 4096, 2048
    w = torch.empty(E, N, K, dtype=torch.float16, device="cuda")
    assert (E - 1) * N * K > 2 ** 31
    w[-1] = _rand(N, K, seed=7)
    for rows in (3, 200):
        x = _rand(rows, K, seed=rows)
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[-1] = rows
        y = g.grouped_linear(x, w, off, out_dtype=torch.float32)
        assert torch.equal(y, x.float() @ w[-1].float().T)
    x = _rand(200, N, seed=9)
    y = g.grouped_linear(x, w, off, opW="N", out_dtype=torch.float32)
    assert torch.equal(y, x.float() @ w[-1].float())


def test_rows_past_32_bits():
    P, H = 600_000, 4096
    assert P * H > 2 ** 31
    x = _rand(P, 64, seed=1)
    w = _rand(1, H, 64, seed=2)
    off = torch.tensor([0, P], dtype=torch.int32, device="cuda")
    y = g.grouped_linear(x, w, off)
    for s in (slice(0, 50), slice(P - 70, P)):
        assert torch.equal(y[s].float(), x[s].float() @ w[0].float().T)
    where = torch.arange(P, dtype=torch.int32, device="cuda").flip(0).reshape(P // 2, 2).contiguous()
    z = g.moe_combine(y, where)
    assert torch.equal(z[0].float(), y[-1].float() + y[-2].float())
    assert torch.equal(z[-1].float(), y[0].float() + y[1].float())
    del z
    back = g.moe_dispatch(y[:P // 2], where)
    assert torch.equal(back[P - 2], y[0]) and torch.equal(back[0], y[P // 2 - 1])


@pytest.mark.parametrize("opW", ["T", "N"])
def test_no_rows_to_read(opW):
    # every position's row is outside an empty x: zeros, and the weights (fewer rows stored than the
    # other op would read) are left alone
    w = _rand(2, 8, 520) if opW == "N" else _rand(2, 520, 8)
    x = torch.empty(0, 8, dtype=torch.float16, device="cuda")
    off = torch.tensor([0, 3, 200], dtype=torch.int32, device="cuda")
    rows = torch.zeros(200, dtype=torch.int32, device="cuda")
    y = g.grouped_linear(x, w, off, rows=rows, opW=opW)
    assert y.shape == (200, 520) and (y == 0).all()


def test_refusals():
    x, w = _rand(8, 16), _rand(2, 24, 16)
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    bad = [
        (ValueError, lambda: g.grouped_linear(x.cpu(), w, off)),
        (TypeError, lambda: g.grouped_linear(x, w.bfloat16(), off)),
        (TypeError, lambda: g.grouped_linear(x, w, off.long())),
        (ValueError, lambda: g.grouped_linear(x, w, off[:2])),
        (ValueError, lambda: g.grouped_linear(x, _rand(2, 24, 8), off)),
        (ValueError, lambda: g.grouped_linear(x, _rand(2, 25, 16), off, gated=True)),
        (ValueError, lambda: g.grouped_linear(x.t(), w, off)),
        (ValueError, lambda: g.grouped_linear(x, w, off, opW="X")),
        (TypeError, lambda: g.grouped_linear(x, w, off, out_dtype=torch.float64)),
        (g.GemmError, lambda: g.grouped_linear(x, w, off, out_dtype=torch.bfloat16)),
        (g.GemmError, lambda: g.grouped_linear(x.float(), w.float(), off)),
        (g.GemmError, lambda: g.grouped_linear(_rand(8, 17)[:, 1:], w, off)),  # rows off 16 bytes
        (ValueError, lambda: g.grouped_weight_grad(x, _rand(7, 16), off)),
        (g.GemmError, lambda: g.grouped_weight_grad(x, _rand(8, 12)[:, :9], off)),
        (ValueError, lambda: g.moe_combine(x, off)),
        (TypeError, lambda: g.moe_combine(x, off.view(1, 3).long())),
        (ValueError, lambda: g.moe_combine(x, off.view(1, 3), torch.ones(1, 2, device="cuda"))),
        (ValueError, lambda: g.moe_route(x[0], 2)),
        (ValueError, lambda: g.moe_route(x, 2, score="cosine")),
        (g.GemmError, lambda: g.moe_route(x, 17)),
        (g.GemmError, lambda: g.moe_route(x, 2, groups=3)),
        (g.GemmError, lambda: g.moe_route(x, 9, groups=2, groups_kept=1)),
        (TypeError, lambda: g.moe_route(x.double(), 2)),
        (ValueError, lambda: g.moe_route(x, 2, bias=torch.zeros(4, device="cuda"))),
        (ValueError, lambda: g.gated_silu_backward(x, x)),
        (ValueError, lambda: g.lora_linear(x, w[0], _rand(2, 8, 16), _rand(2, 24, 4), off, off[:2])),
        (ValueError, lambda: g.lora_linear(x, w[0], _rand(2, 8, 16), _rand(2, 24, 8), off[:2], off[:2])),
        (g.GemmError, lambda: g.lora_linear(x, w[0], _rand(2, 136, 16), _rand(2, 24, 136), off, off[:2])),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
    assert torch.equal(g.grouped_linear(x, w, off, out_dtype=torch.float32)[:4], x[:4].float() @ w[0].float().T)


@pytest.mark.parametrize("T", [40, 300])
def test_split_sums_and_requests(T):
    # K long and few tiles: parts of K and of the requests' slices are summed by a second kernel
    gen = torch.Generator().manual_seed(T)
    N, K, R, Q = 136, 4104, 24, 11
    x, w = torch.randn(T, K, generator=gen).bfloat16(), (torch.randn(N, K, generator=gen) * K ** -0.5).bfloat16()
    a = (torch.randn(5, R, K, generator=gen) * K ** -0.5).bfloat16()
    b = (torch.randn(5, N, R, generator=gen) * R ** -0.5).bfloat16()
    cuts = torch.cat([torch.tensor([0]), torch.sort(torch.randint(0, T + 1, (Q - 1,), generator=gen)).values, torch.tensor([T])])
    who = torch.randint(-1, 5, (Q,), generator=gen)
    y = g.lora_linear(x.cuda(), w.cuda(), a.cuda(), b.cuda(), cuts.int().cuda(), who.int().cuda(), out_dtype=torch.float32)
    want = x.double() @ w.double().T
    size = x.double().abs() @ w.double().abs().T
    for q in range(Q):
        s, i = slice(int(cuts[q]), int(cuts[q + 1])), int(who[q])
        if i >= 0:
            want[s] += x[s].double() @ a[i].double().T @ b[i].double().T
            size[s] += x[s].double().abs() @ a[i].double().abs().T @ b[i].double().abs().T
    ref.assert_within(y, want, (ref.sum_bound(K) + (R + 4) * 2.0 ** -23) * size)
