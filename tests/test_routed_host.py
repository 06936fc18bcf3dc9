"""Host-side checks of the routed products that need no GPU: every entry point validates its arguments
before touching a device."""
import pytest

import dense_gemm_sgemm_gb300 as g
from dense_gemm_sgemm_gb300 import _lib, build

P = 4096  # a fake, never dereferenced address: every call below returns before any launch
OK, INVALID, MISALIGNED, UNSUPPORTED = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _call(fn, defaults, **changes):
    args = dict(defaults)
    assert set(changes) <= set(args), set(changes) - set(args)
    args.update(changes)
    return fn(*args.values())


ROUTE = dict(type=0, T=4, E=8, logits=P, ld=8, bias=None, score=0, groups=1, kept=1, top=1, k=2, renorm=1, scale=1.0,
             ids=P, weights=P, offsets=P, tokens=P, where=P, stream=None)


@pytest.mark.parametrize("status,changes", [
    (INVALID, dict(type=3)), (INVALID, dict(score=2)), (INVALID, dict(T=-1)), (INVALID, dict(E=0)), (INVALID, dict(k=0)),
    (INVALID, dict(k=9)), (INVALID, dict(ld=7)), (INVALID, dict(groups=3)), (INVALID, dict(groups=0)),
    (INVALID, dict(groups=4, kept=5)), (INVALID, dict(groups=4, kept=1, k=3)), (INVALID, dict(top=3)),
    (INVALID, dict(logits=None)), (INVALID, dict(ids=None)), (INVALID, dict(tokens=None)), (INVALID, dict(offsets=None)),
    (UNSUPPORTED, dict(E=1025, ld=1025)), (UNSUPPORTED, dict(E=64, ld=64, groups=64, kept=64)),
    (UNSUPPORTED, dict(E=64, ld=64, k=33)), (UNSUPPORTED, dict(T=1 << 30)),
    (MISALIGNED, dict(logits=P + 2)), (MISALIGNED, dict(ids=P + 1)), (MISALIGNED, dict(type=1, logits=P + 1)),
    (OK, dict(T=0, offsets=None, tokens=None, where=None)),
])
def test_route(lib, status, changes):
    assert _call(lib.gemm_moe_route, ROUTE, **changes) == status


LINEAR = dict(type=1, y_type=1, groups=2, offsets=P, op=1, gated=0, N=8, K=16, X=P, ldx=16, x_rows=10, rows=None, W=P,
              ldw=16, strideW=128, Y=P, ldy=8, y_rows=10, pre=None, ldp=0, work=None, stream=None)


@pytest.mark.parametrize("status,changes", [
    (INVALID, dict(type=0)), (INVALID, dict(y_type=2)), (INVALID, dict(op=2)), (INVALID, dict(op=0, gated=1)),
    (INVALID, dict(pre=P, ldp=16)), (INVALID, dict(ldx=15)), (INVALID, dict(ldw=8)), (INVALID, dict(ldy=4)),
    (INVALID, dict(gated=1, pre=P, ldp=8)), (INVALID, dict(offsets=None)), (INVALID, dict(W=None)), (INVALID, dict(X=None)),
    (INVALID, dict(Y=None)), (INVALID, dict(strideW=120)), (INVALID, dict(groups=-1)), (INVALID, dict(x_rows=-1)),
    (UNSUPPORTED, dict(groups=1025)), (UNSUPPORTED, dict(K=1 << 24, ldx=1 << 24, ldw=1 << 24)),
    (UNSUPPORTED, dict(y_rows=1 << 31)),
    (MISALIGNED, dict(X=P + 8)), (MISALIGNED, dict(ldx=20)), (MISALIGNED, dict(ldw=20, strideW=160)),
    (MISALIGNED, dict(strideW=132)), (MISALIGNED, dict(Y=P + 2)), (MISALIGNED, dict(ldy=12)), (MISALIGNED, dict(work=P + 8)),
    (MISALIGNED, dict(rows=P + 2)), (OK, dict(y_rows=0)), (OK, dict(groups=0)), (OK, dict(N=0, ldy=8)),
])
def test_grouped_linear(lib, status, changes):
    assert _call(lib.gemm_grouped_linear, LINEAR, **changes) == status


GRAD = dict(type=2, dw_type=0, groups=2, offsets=P, N=8, K=16, dY=P, lddy=8, X=P, ldx=16, positions=5, dW=P, lddw=16,
            strideDW=128, stream=None)


@pytest.mark.parametrize("status,changes", [
    (INVALID, dict(type=0)), (INVALID, dict(dw_type=1)), (INVALID, dict(lddy=4)), (INVALID, dict(lddw=8)),
    (INVALID, dict(strideDW=120)), (INVALID, dict(X=None)), (INVALID, dict(dW=None)), (INVALID, dict(positions=-1)),
    (UNSUPPORTED, dict(groups=1025)), (MISALIGNED, dict(lddy=12)), (MISALIGNED, dict(dW=P + 4)),
    (MISALIGNED, dict(strideDW=132)), (OK, dict(K=0, ldx=16)), (OK, dict(groups=0)),
])
def test_grouped_weight_grad(lib, status, changes):
    assert _call(lib.gemm_grouped_weight_grad, GRAD, **changes) == status


LORA = dict(type=1, y_type=1, T=4, N=8, K=16, X=P, ldx=16, W=P, ldw=16, requests=2, segments=P, adapters=P, count=3, R=8,
            A=P, lda=16, strideA=128, B=P, ldb=8, strideB=64, scales=None, Y=P, ldy=8, work=P, stream=None)


@pytest.mark.parametrize("status,changes", [
    (INVALID, dict(type=0)), (INVALID, dict(y_type=2)), (INVALID, dict(lda=8)), (INVALID, dict(ldb=4)),
    (INVALID, dict(segments=None)), (INVALID, dict(work=None)), (INVALID, dict(A=None)), (INVALID, dict(W=None)),
    (INVALID, dict(R=-1)), (UNSUPPORTED, dict(R=129, ldb=136)), (UNSUPPORTED, dict(T=1 << 24)),
    (UNSUPPORTED, dict(requests=12_000_000)), (MISALIGNED, dict(work=P + 8)), (MISALIGNED, dict(ldb=12)),
    (MISALIGNED, dict(strideA=132)), (MISALIGNED, dict(X=P + 2)), (MISALIGNED, dict(scales=P + 2)), (OK, dict(T=0)),
])
def test_lora_linear(lib, status, changes):
    assert _call(lib.gemm_lora_linear, LORA, **changes) == status


def test_lora_work_bytes(lib):
    f = lib.gemm_lora_work_bytes
    assert f(0, 8, 8, 1, 8) == 0 and f(4, 8, 8, 0, 8) == 0 and f(4, 8, 8, 1, 0) == 0 and f(4, 8, 8, 1, 129) == 0
    for T, N, K, Q, R in ((1, 8, 8, 1, 1), (100, 4096, 4096, 64, 16), (8192, 4096, 4096, 7, 64), (300, 24, 4096, 3, 128)):
        n = f(T, N, K, Q, R)
        assert n % 16 == 0
        assert n >= 4 * T * (R + 1)                                     # fp32 inner products and adapter numbers
        assert n >= (T // 32 + Q) * 32 * 128 * 3 * ((R + 63) // 64)     # three 16-bit parts of 64 ranks


def test_row_movement_and_activation(lib):
    d, c, b, s = lib.gemm_moe_dispatch, lib.gemm_moe_combine, lib.gemm_moe_combine_backward, lib.gemm_gated_silu_backward
    assert d(0, 4, 8, 2, P, 8, P, None, 8, P, 7, None) == INVALID
    assert d(0, 4, 8, 2, None, 8, P, None, 8, P, 8, None) == INVALID
    assert d(1, 4, 8, 2, P + 1, 8, P, None, 8, P, 8, None) == MISALIGNED
    assert d(0, 0, 8, 2, None, 8, None, None, 8, None, 8, None) == OK
    assert c(0, 5, 4, 8, 2, P, 8, 8, P, None, P, 8, None) == INVALID
    assert c(0, 0, 4, 8, 0, P, 8, 8, P, None, P, 8, None) == INVALID
    assert c(0, 0, 4, 8, 2, P, 8, 8, P, None, P + 2, 8, None) == MISALIGNED
    assert c(0, 0, 1 << 31, 8, 2, P, 8, 8, P, None, P, 8, None) == UNSUPPORTED
    assert b(1, 0, 4, 8, 2, P, 8, P, 8, 8, P, P, P, 8, None, None) == INVALID
    assert b(1, 0, 4, 8, 2, P, 8, P, 4, 8, P, P, P, 8, P, None) == INVALID
    assert s(0, 0, 4, 8, P, 16, P, 8, P, 16, None) == INVALID      # fp32 pre
    assert s(1, 2, 4, 8, P, 16, P, 8, P, 16, None) == INVALID      # dh of another 16-bit type
    assert s(1, 1, 4, 8, P, 15, P, 8, P, 16, None) == INVALID
    assert s(1, 1, 0, 8, None, 16, None, 8, None, 16, None) == OK
    plan = lib.gemm_moe_plan
    assert plan(4, 8, 2, None, P, P, P, None) == INVALID
    assert plan(4, 0, 2, P, P, P, P, None) == INVALID
    assert plan(4, 8, 1025, P, P, P, P, None) == UNSUPPORTED
    assert plan(4, 8, 2, P + 2, P, P, P, None) == MISALIGNED


def test_tensor_calls_refuse_what_is_no_cuda_tensor(lib):
    import torch

    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        g.moe_route(x, 2)
    with pytest.raises(TypeError):
        g.moe_route([[1.0]], 1)
    with pytest.raises(ValueError):
        g.grouped_linear(x.half(), torch.zeros(1, 8, 8).half(), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        g.lora_linear(x.half(), x.half(), x.half(), x.half(), x, x)
