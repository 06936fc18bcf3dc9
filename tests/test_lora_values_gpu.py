"""Adapters whose values, or whose inner products, leave the ordinary range: one request's infinities and
NaN stay in its own tokens, whichever form of the layer takes the call."""
import math

import pytest
import torch

import dense_gemm_sgemm_gb300 as g
from tests import routed_reference as ref

pytestmark = pytest.mark.gpu

# up to 64 tokens the few-rows form takes the call, beyond it the tcgen05 form
BATCHES = {
    "few": ([1, 1, 20, 1, 30], [0, -1, 1, 0, 2]),
    "shared blocks": ([1, 1, 60, 1, 100, 7], [0, -1, 1, 2, 0, 1]),
    "single tokens": ([1] * 150, [i % 5 - 1 for i in range(150)]),
    "long prompts": ([300, 290, 5], [1, 0, 2]),
}


def _reference(c, R):
    """y in 64 bits by the formula (its infinities and NaN included), the bound where it is finite, and
    where the sign of an infinity is beyond the inner products' rounding."""
    x, w = c["x"].double(), c["w"].double()
    K = x.shape[1]
    y, bound = x @ w.T, ref.sum_bound(K) * (x.abs() @ w.abs().T)
    sure = torch.ones_like(y, dtype=torch.bool)
    seg = c["segments"].tolist()
    for q, i in enumerate(c["adapters"].tolist()):
        if i < 0:
            continue
        s = slice(seg[q], seg[q + 1])
        a, b = c["a"][i].double(), c["b"][i].double()
        inner = x[s] @ a.T
        size = x[s].abs() @ a.abs().nan_to_num(0.0, 0.0, 0.0).T
        y[s] += inner @ b.T
        sure[s] = (inner.nan_to_num(1.0, 1.0, 1.0).abs() > ref.sum_bound(K) * size + 2.0 ** -20).all(1, keepdim=True)
        bound[s] += (ref.sum_bound(K) + (R + 4) * 2.0 ** -23) * (size @ b.abs().nan_to_num(0.0, 0.0, 0.0).T)
        bound[s] += (R + 4) * 2.0 ** -23 * y[s].abs().nan_to_num(0.0, 0.0, 0.0)
    return y, bound, sure


def _case(lengths, who, R, N, K, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).to(dtype)  # noqa: E731
    c = {"x": rnd(sum(lengths), K), "w": rnd(N, K, std=K ** -0.5), "a": rnd(4, R, K, std=K ** -0.5),
         "b": rnd(4, N, R, std=R ** -0.5)}
    c["segments"] = torch.cat([torch.zeros(1, dtype=torch.long), torch.tensor(lengths).cumsum(0)]).int()
    c["adapters"] = torch.tensor(who, dtype=torch.int32)
    return c


def _pad(t):
    wide = torch.zeros(*t.shape[:-1], (t.shape[-1] + 7) // 8 * 8, dtype=t.dtype)
    wide[..., :t.shape[-1]] = t
    return wide.cuda()[..., :t.shape[-1]]


def _run(c, out_dtype=None):
    y = g.lora_linear(_pad(c["x"]), _pad(c["w"]), _pad(c["a"]), _pad(c["b"]), c["segments"].cuda(), c["adapters"].cuda(),
                      out_dtype=out_dtype)
    assert g.gemm_get_device_status() == 0
    return y.cpu()


def _check(c, R, out_dtype=None):
    y, (want, bound, sure) = _run(c, out_dtype), _reference(c, R)
    finite = torch.isfinite(want)
    leaked = finite & ~torch.isfinite(y.double())
    assert not leaked.any(), f"{int(leaked.sum())} finite values lost, first at {leaked.nonzero()[0].tolist()}"
    ref.assert_within(torch.where(finite, y, 0.0).to(y.dtype), torch.where(finite, want, 0.0), bound)
    assert not torch.isfinite(y[~finite]).any()
    exact = ~finite & sure
    assert torch.equal(torch.nan_to_num(y[exact].double(), 0.0, 1.0, -1.0), torch.nan_to_num(want[exact], 0.0, 1.0, -1.0))


@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("which,value", [("b", math.inf), ("b", -math.inf), ("b", math.nan), ("a", math.inf), ("a", math.nan)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_an_adapters_infinities_stay_with_its_tokens(batch, which, value, dtype):
    lengths, who = BATCHES[batch]
    for R, N, K in ((16, 600, 200), (5, 72, 64), (100, 264, 72)):
        c = _case(lengths, who, R, N, K, dtype, seed=R)
        # one element, in a feature of the last tile of 256 and in the last rank
        c[which][0, N - 3 if which == "b" else R - 1, R - 1 if which == "b" else 7] = value
        _check(c, R, torch.float32 if R == 5 else None)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_infinities_where_k_is_split(dtype):
    # few tiles and a long K: parts of K and of the requests summed by a second kernel
    c = _case([1] * 90 + [40, 3], [i % 5 - 1 for i in range(92)], 24, 136, 4104, dtype)
    c["b"][3, 100, 2] = math.inf
    c["b"][1, 7, 23] = math.nan
    _check(c, 24, torch.float32)


def test_many_requests_of_bad_adapters():
    # every adapter has an infinity, each in another feature, some features in none
    c = _case([3] * 70, [i % 4 for i in range(70)], 16, 520, 128, torch.float16)
    for i in range(4):
        c["b"][i, 130 * i, i] = math.inf
    _check(c, 16, torch.float32)


@pytest.mark.parametrize("T,requests,R", [(4096, 3, 64), (2048, 2048, 128)])
def test_whole_batches_of_bad_values_expire_no_wait(T, requests, R):
    # every tile is computed twice, with every request's product on the CUDA cores
    H = 1024
    x, w = torch.randn(T, H, device="cuda").half(), torch.randn(H, H, device="cuda").half()
    a, b = torch.randn(4, R, H, device="cuda").half(), torch.randn(4, H, R, device="cuda").half()
    b[:, ::7, R // 2] = math.inf
    cuts = torch.linspace(0, T, requests + 1, device="cuda").round().int()
    who = torch.arange(requests, device="cuda", dtype=torch.int32) % 4
    y = g.lora_linear(x, w, a, b, cuts, who)
    assert g.gemm_get_device_status() == 0
    bad = torch.zeros(H, dtype=torch.bool, device="cuda")
    bad[::7] = True
    assert torch.isfinite(y[:, ~bad]).all() and not torch.isfinite(y[:, bad]).any()
    x[:] = math.nan
    assert torch.isnan(g.lora_linear(x, w, a, b, cuts, who)).all()
    assert g.gemm_get_device_status() == 0


@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("out_dtype", [torch.float16, torch.float32])
def test_inner_products_beyond_fp16(batch, out_dtype):
    # inner products of about 10^5, on both sides of fp16's largest, times small B: ordinary results
    lengths, who = BATCHES[batch]
    for R in (8, 40, 128):
        c = _case(lengths, who, R, 264, 200, torch.float16, seed=R)
        c["a"][0] *= 20000.0
        c["x"] *= 4.0
        c["b"] *= 2.0 ** -9
        seg = c["segments"].tolist()
        inner = torch.cat([c["x"][seg[q]:seg[q + 1]].double() @ c["a"][0].double().T for q, i in enumerate(who) if i == 0])
        assert (inner.abs() > 65520).any() and (inner.abs() < 65504).any()
        _check(c, R, out_dtype)


@pytest.mark.parametrize("tokens", [3, 100])
def test_inner_products_beyond_bf16(tokens):
    # fp32 values above bf16's largest: inner = scale
    x = torch.ones(tokens, 8, dtype=torch.bfloat16)
    x[:, 1:] = 0.0
    a, b = torch.zeros(1, 8, 8, dtype=torch.bfloat16), torch.zeros(1, 40, 8, dtype=torch.bfloat16)
    a[0, 2, 0], b[0, :, 2] = 1.0, 2.0 ** -120
    w = torch.zeros(40, 8, dtype=torch.bfloat16)
    scale = torch.tensor([3.4e38])
    y = g.lora_linear(x.cuda(), w.cuda(), a.cuda(), b.cuda(), torch.tensor([0, tokens], dtype=torch.int32, device="cuda"),
                      torch.zeros(1, dtype=torch.int32, device="cuda"), scales=scale.cuda(), out_dtype=torch.float32)
    assert torch.equal(y.cpu(), (scale * 2.0 ** -120).expand(tokens, 40))


@pytest.mark.parametrize("dtype,out_dtype", [(torch.float16, torch.float32), (torch.bfloat16, torch.float32),
                                             (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("tokens", [40, 130])
def test_precision_of_the_inner_products(dtype, out_dtype, tokens):
    # x = a = b = 1 and one adapter a token: the outputs are the inner products, which are the scales
    gen = torch.Generator().manual_seed(tokens)
    scales = torch.exp2(torch.rand(tokens, generator=gen) * 31 - 16) * torch.where(torch.rand(tokens, generator=gen) < 0.5, -1, 1)
    one = torch.ones(tokens, 8, 8, dtype=dtype, device="cuda")[..., :1]
    y = g.lora_linear(one[:, 0], torch.zeros(8, 8, dtype=dtype, device="cuda")[:, :1], one[:, :1], one,
                      torch.arange(tokens + 1, dtype=torch.int32, device="cuda"),
                      torch.arange(tokens, dtype=torch.int32, device="cuda"), scales=scales.cuda(), out_dtype=out_dtype)
    v = scales.double().abs()
    if tokens <= 64:
        bound = torch.zeros_like(v)  # fp32
    elif dtype is torch.float16:
        bound = torch.maximum(v * 2.0 ** -22, torch.tensor(2.0 ** -25))
    else:
        bound = v * (2.0 ** -24 if out_dtype is torch.float32 else 2.0 ** -16)
    ref.assert_within(y.cpu(), scales.double()[:, None].expand(-1, 8), bound[:, None].expand(-1, 8))
