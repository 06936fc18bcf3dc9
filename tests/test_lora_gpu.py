"""A shared linear layer with adapters of many requests against a plain 64-bit form."""
import math

import pytest
import torch

import dense_gemm_sgemm_gb300 as g
from tests import routed_reference as ref

pytestmark = pytest.mark.gpu


def _case(lengths, who, count, R, N, K, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    T = sum(lengths)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).to(dtype)  # noqa: E731
    c = {"x": rnd(T, K), "w": rnd(N, K, std=K ** -0.5), "a": rnd(count, R, K, std=K ** -0.5),
         "b": rnd(count, N, R, std=max(R, 1) ** -0.5), "scales": torch.rand(count, generator=gen) + 0.5}
    c["segments"] = torch.cat([torch.zeros(1, dtype=torch.long), torch.tensor(lengths).cumsum(0)]).int()
    c["adapters"] = torch.tensor(who, dtype=torch.int32)
    return c


def _reference(c, scaled=True):
    x, w, R = c["x"].double(), c["w"].double(), c["a"].shape[1]
    K = x.shape[1]
    y = x @ w.T
    bound = ref.sum_bound(K) * (x.abs() @ w.abs().T)
    seg = c["segments"].tolist()
    for q, i in enumerate(c["adapters"].tolist()):
        if not 0 <= i < c["a"].shape[0]:
            continue
        s = slice(max(seg[q], 0), min(seg[q + 1], x.shape[0]))
        f = c["scales"][i].double() if scaled else 1.0
        a, b = c["a"][i].double(), c["b"][i].double()
        inner, size = f * x[s] @ a.T, f * x[s].abs() @ a.abs().T
        y[s] += inner @ b.T
        # the inner product's own error, and the R further terms of the outer sum
        bound[s] += (ref.sum_bound(K) + (R + 4) * 2.0 ** -23) * (size @ b.abs().T)
        bound[s] += (R + 4) * 2.0 ** -23 * y[s].abs()
    return y, bound


def _pad(t, extra):
    wide = torch.full((*t.shape[:-1], t.shape[-1] + (-t.shape[-1]) % 8 + extra), math.nan, dtype=t.dtype)
    wide[..., :t.shape[-1]] = t
    return wide.cuda()[..., :t.shape[-1]]


def _check(c, extra=0, scaled=True, out_dtype=None):
    y = g.lora_linear(_pad(c["x"], extra), _pad(c["w"], extra), _pad(c["a"], extra), _pad(c["b"], extra),
                      c["segments"].cuda(), c["adapters"].cuda(),
                      scales=c["scales"].cuda() if scaled else None, out_dtype=out_dtype)
    assert g.gemm_get_device_status() == 0
    ref.assert_within(y, *_reference(c, scaled))
    return y


CASES = {
    "one token": ([1], [0]),
    "one token without adapter": ([1], [-1]),
    "single tokens": ([1] * 37, [i % 7 - 1 for i in range(37)]),
    "empty requests": ([0, 3, 0, 0, 5, 0], [1, 0, 2, 3, 3, 1]),
    "prompts": ([70, 1, 200, 33, 129], [2, 0, -1, 1, 2]),
    "one long prompt": ([517], [4]),
    "mixed": ([1] * 20 + [90] + [1] * 5 + [31, 64], [i % 6 for i in range(28)]),
    "adapters out of range": ([4, 4, 80, 2], [7, 1, 99, -5]),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("R", [8, 16, 24, 64])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_requests(name, R, dtype):
    lengths, who = CASES[name]
    _check(_case(lengths, who, 7, R, 264, 200, dtype, seed=R))


@pytest.mark.parametrize("N,K", [(1, 1), (7, 65), (129, 8), (1001, 513), (256, 2048)])
@pytest.mark.parametrize("R", [1, 5, 33, 100, 128])
def test_odd_sizes(N, K, R):
    _check(_case([3, 0, 1, 40], [0, 1, 2, 1], 3, R, N, K, torch.bfloat16, seed=N), extra=8, out_dtype=torch.float32)
    _check(_case([150, 1, 99], [2, 0, 1], 3, R, N, K, torch.float16, seed=K), scaled=False)


def test_nothing_beside_the_projection():
    for count, R, requests in ((0, 8, 2), (2, 0, 2), (2, 8, 0)):
        c = _case([5, 6], [0, 1], count, R, 40, 48, torch.float16)
        c["adapters"], c["segments"] = c["adapters"][:requests], c["segments"][:requests + 1]
        if count == 0 or R == 0:
            want = c["x"].double() @ c["w"].double().T
            size = c["x"].double().abs() @ c["w"].double().abs().T
            y = g.lora_linear(c["x"].cuda(), c["w"].cuda(), c["a"].cuda(), c["b"].cuda(), c["segments"].cuda(),
                              c["adapters"].cuda())
            ref.assert_within(y, want, ref.sum_bound(48) * size)
        else:
            _check(c)


def test_tokens_outside_every_request():
    # requests cover tokens 4 .. 10 of 90 only; bounds past the tokens are clamped
    c = _case([4, 7, 79], [-1, 2, -1], 3, 16, 72, 64, torch.bfloat16)
    want = _reference(c)
    c["segments"], c["adapters"] = c["segments"][1:3].clone(), c["adapters"][1:2].clone()
    y = g.lora_linear(c["x"].cuda(), c["w"].cuda(), c["a"].cuda(), c["b"].cuda(), c["segments"].cuda(),
                      c["adapters"].cuda(), scales=c["scales"].cuda())
    ref.assert_within(y, *want)
    c["segments"] = torch.tensor([-3, 2 ** 30], dtype=torch.int32)
    _check(c)


def test_other_requests_values_stay_there():
    c = _case([1, 1, 60, 1, 100], [0, 1, 2, 1, 0], 3, 16, 72, 64, torch.float16)
    want = _check(c)
    c["x"][1] = math.nan
    c["x"][62] = math.inf
    y = g.lora_linear(*(c[n].cuda() for n in ("x", "w", "a", "b", "segments", "adapters")), scales=c["scales"].cuda())
    keep = torch.ones(163, dtype=torch.bool)
    keep[1], keep[62] = False, False
    assert torch.equal(y[keep.cuda()], want[keep.cuda()]) and torch.isnan(y[1]).all()


def test_calls_in_a_row_do_not_share_their_work():
    # the inner products of one call are not seen by the next, on one stream or on two
    cs = [_case([1] * 50, [i % 5 for i in range(50)], 5, 16, 512, 256, torch.float16, seed=s) for s in range(4)]
    dev = [[c[n].cuda() for n in ("x", "w", "a", "b", "segments", "adapters")] for c in cs]
    alone = []
    for d in dev:
        alone.append(g.lora_linear(*d))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        out = []
        for i, d in enumerate(dev):
            with torch.cuda.stream(streams[i % 2]):
                out.append(g.lora_linear(*d))
        torch.cuda.synchronize()
        for o, a in zip(out, alone):
            assert torch.equal(o, a)
