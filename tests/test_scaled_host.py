"""Host-side checks of the block-scaled products and the orthogonalised update that need no GPU: every entry
point validates its arguments before touching a device."""
import ctypes

import pytest

import dense_gemm_sgemm_gb300 as g
from dense_gemm_sgemm_gb300 import _lib, build

P = 4096  # a fake, never dereferenced address: every call below returns before any launch
OK, INVALID, MISALIGNED, UNSUPPORTED = 0, 1, 2, 3
E4M3, E5M2 = 3, 4


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _call(fn, defaults, **changes):
    args = dict(defaults)
    assert set(changes) <= set(args), set(changes) - set(args)
    args.update(changes)
    return fn(*args.values())


QUANTIZE = dict(type=2, q_type=E4M3, rows=10, cols=40, X=P, ldx=40, block_rows=1, block_cols=128, Q=P, ldq=48, scales=P, s_row=1,
                s_col=10, stream=None)


@pytest.mark.parametrize("status,changes", [
    (INVALID, dict(type=E4M3)), (INVALID, dict(type=9)), (INVALID, dict(q_type=2)), (INVALID, dict(rows=-1)), (INVALID, dict(cols=-1)),
    (INVALID, dict(ldx=39)), (INVALID, dict(ldq=32)), (INVALID, dict(block_rows=1, block_cols=1)), (INVALID, dict(block_rows=2)),
    (INVALID, dict(block_cols=64)), (INVALID, dict(block_rows=0)), (INVALID, dict(X=None)), (INVALID, dict(Q=None)),
    (INVALID, dict(scales=None)), (INVALID, dict(s_row=-1)), (INVALID, dict(s_col=-1)), (UNSUPPORTED, dict(rows=1 << 30)),
    (UNSUPPORTED, dict(cols=1 << 30, ldx=1 << 30, ldq=1 << 30)), (UNSUPPORTED, dict(ldx=1 << 36)), (UNSUPPORTED, dict(s_row=1 << 41)),
    (MISALIGNED, dict(X=P + 1)), (MISALIGNED, dict(type=0, X=P + 2)), (MISALIGNED, dict(Q=P + 8)), (MISALIGNED, dict(ldq=44)),
    (MISALIGNED, dict(scales=P + 2)), (MISALIGNED, dict(block_rows=128, block_cols=1, Q=P + 8)),
    (OK, dict(rows=0)), (OK, dict(cols=0)), (OK, dict(rows=0, X=None, Q=None, scales=None)),
])
def test_quantize_blocks(lib, status, changes):
    assert _call(lib.gemm_quantize_blocks, QUANTIZE, **changes) == status


BOTH = dict(type=2, q_type=E5M2, rows=10, cols=40, X=P, ldx=40, Q=P, ldq=48, scales=P, s_row=1, s_col=10, Qc=P, ldqc=48, scales_c=P,
            sc_row=40, sc_col=1, stream=None)


@pytest.mark.parametrize("status,changes", [
    (INVALID, dict(type=5)), (INVALID, dict(q_type=0)), (INVALID, dict(Q=None)), (INVALID, dict(Qc=None)), (INVALID, dict(scales=None)),
    (INVALID, dict(scales_c=None)), (INVALID, dict(ldqc=39)), (INVALID, dict(sc_row=-1)), (UNSUPPORTED, dict(rows=1 << 30)),
    (MISALIGNED, dict(Qc=P + 4)), (MISALIGNED, dict(ldqc=50)), (MISALIGNED, dict(scales_c=P + 1)), (OK, dict(rows=0)), (OK, dict(cols=0)),
])
def test_quantize_both(lib, status, changes):
    assert _call(lib.gemm_quantize_both, BOTH, **changes) == status


BACK = dict(q_type=E4M3, y_type=2, rows=10, cols=40, Q=P, ldq=48, block_rows=1, block_cols=128, scales=P, s_row=1, s_col=10, Y=P, ldy=40,
            stream=None)


@pytest.mark.parametrize("status,changes", [
    (INVALID, dict(q_type=1)), (INVALID, dict(y_type=E5M2)), (INVALID, dict(block_rows=1, block_cols=1)), (INVALID, dict(Q=None)),
    (INVALID, dict(Y=None)), (INVALID, dict(scales=None)), (INVALID, dict(ldy=39)), (INVALID, dict(ldq=39)),
    (UNSUPPORTED, dict(rows=1 << 30)), (MISALIGNED, dict(Q=P + 1)), (MISALIGNED, dict(ldq=40)), (MISALIGNED, dict(Y=P + 1)),
    (OK, dict(rows=0)), (OK, dict(cols=0)),
])
def test_dequantize_blocks(lib, status, changes):
    assert _call(lib.gemm_dequantize_blocks, BACK, **changes) == status


MATMUL = dict(a_type=E4M3, b_type=E5M2, c_type=2, opA=0, opB=1, M=10, N=20, K=300, A=P, lda=304, a_block=1, a_scales=P, sa_row=1, sa_col=10,
              B=P, ldb=304, b_block=128, b_scales=P, sb_row=3, sb_col=1, C=P, ldc=24, stream=None)


@pytest.mark.parametrize("status,changes", [
    (INVALID, dict(a_type=2)), (INVALID, dict(b_type=0)), (INVALID, dict(c_type=E4M3)), (INVALID, dict(opA=2)), (INVALID, dict(opB=-1)),
    (INVALID, dict(a_block=64)), (INVALID, dict(b_block=0)), (INVALID, dict(M=-1)), (INVALID, dict(K=-1)), (INVALID, dict(lda=288)),
    (INVALID, dict(opA=1, lda=9)), (INVALID, dict(opB=0, ldb=19)), (INVALID, dict(ldc=19)), (INVALID, dict(A=None)), (INVALID, dict(B=None)),
    (INVALID, dict(C=None)), (INVALID, dict(a_scales=None)), (INVALID, dict(b_scales=None)), (INVALID, dict(sa_row=-1)),
    (UNSUPPORTED, dict(M=1 << 30)), (UNSUPPORTED, dict(N=1 << 30, ldc=1 << 30)), (UNSUPPORTED, dict(K=1 << 30, lda=1 << 30, ldb=1 << 30)),
    (UNSUPPORTED, dict(sb_col=1 << 41)), (MISALIGNED, dict(A=P + 8)), (MISALIGNED, dict(lda=308)), (MISALIGNED, dict(B=P + 1)),
    (MISALIGNED, dict(ldb=312 + 4)), (MISALIGNED, dict(C=P + 8)), (MISALIGNED, dict(ldc=20)), (MISALIGNED, dict(a_scales=P + 2)),
    (OK, dict(M=0)), (OK, dict(N=0)), (OK, dict(M=0, A=None, a_scales=None, C=None)),
])
def test_scaled_matmul(lib, status, changes):
    assert _call(lib.gemm_scaled_matmul, MATMUL, **changes) == status


def triples(*values):
    return (ctypes.c_float * len(values))(*values)


UPDATE = dict(type=0, y_type=2, count=2, rows=10, cols=20, G=P, ldg=20, strideG=200, steps=2,
              coefficients=triples(3.4445, -4.7750, 2.0315, 1.5, -0.5, 0.0), eps=1e-7, Y=P, ldy=24, strideY=240, work=P, stream=None)


@pytest.mark.parametrize("status,changes", [
    (INVALID, dict(type=E4M3)), (INVALID, dict(y_type=7)), (INVALID, dict(count=-1)), (INVALID, dict(rows=-1)), (INVALID, dict(ldg=19)),
    (INVALID, dict(ldy=16)), (INVALID, dict(steps=0)), (INVALID, dict(coefficients=None)), (INVALID, dict(eps=-1.0)),
    (INVALID, dict(eps=float("nan"))), (INVALID, dict(eps=float("inf"))), (INVALID, dict(strideG=-1)), (INVALID, dict(strideY=200)),
    (INVALID, dict(G=None)), (INVALID, dict(Y=None)), (INVALID, dict(work=None)),
    (UNSUPPORTED, dict(count=1 << 16)), (UNSUPPORTED, dict(rows=1 << 20)), (UNSUPPORTED, dict(cols=1 << 20, ldg=1 << 20, ldy=1 << 20)),
    (UNSUPPORTED, dict(steps=65, coefficients=triples(*[0.5, 0.0, 0.0] * 65))), (UNSUPPORTED, dict(strideY=1 << 41)),
    # growing without bound; not finite
    (UNSUPPORTED, dict(coefficients=triples(300.0, 0.0, 0.0, 300.0, 0.0, 0.0))),
    (UNSUPPORTED, dict(coefficients=triples(2.0, float("nan"), 0.0, 1.0, 0.0, 0.0))),
    (UNSUPPORTED, dict(coefficients=triples(2.0, float("inf"), 0.0, 1.0, 0.0, 0.0))),
    (MISALIGNED, dict(G=P + 2)), (MISALIGNED, dict(Y=P + 8)), (MISALIGNED, dict(ldy=20)), (MISALIGNED, dict(strideY=244)),
    (MISALIGNED, dict(work=P + 128)), (OK, dict(count=0)), (OK, dict(rows=0)), (OK, dict(cols=0)),
])
def test_orthogonalize(lib, status, changes):
    assert _call(lib.gemm_orthogonalize, UPDATE, **changes) == status


def test_work_bytes(lib):
    of = lib.gemm_orthogonalize_work_bytes
    assert of(0, 5, 5) == of(1, 0, 5) == of(1, 5, 0) == of(-1, 5, 5) == of(1, 1 << 20, 5) == 0
    assert of(1, 100, 200) == of(1, 200, 100)  # the smaller side decides, whichever it is
    # two sets of two fp16 parts of X, two parts of E and of F, rows padded to 64
    assert of(3, 100, 200) >= 3 * (2 * 2 * 100 * 256 * 2 + 2 * 2 * 100 * 128 * 2)
    assert of(1, 4096, 4096) < 17 * 4096 * 4096


def test_refusals_of_the_tensor_level():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 256)
    q, s = torch.zeros(4, 256, dtype=torch.float8_e4m3fn), torch.ones(4, 2)
    for call in (lambda: g.quantize_blocks(x), lambda: g.quantize_both(x), lambda: g.dequantize_blocks(q, s),
                 lambda: g.scaled_matmul(q, s, q, s), lambda: g.orthogonalize(x)):
        with pytest.raises(ValueError, match="CUDA"):  # no silent fallback to the host
            call()
    for block in ((1, 1), (2, 128), (128,), (64, 64)):
        with pytest.raises(ValueError, match="block"):
            g.quantize_blocks(x, block)
    with pytest.raises(ValueError, match="opA"):
        g.scaled_matmul(q, s, q, s, opA="X")
    with pytest.raises(TypeError):
        g.quantize_blocks("x")
    with pytest.raises(ValueError, match="three"):
        g.orthogonalize(x, steps=2, coefficients=((1.0, 2.0), (1.0, 2.0)))


def test_names_are_in_the_package_and_their_modules():
    pytest.importorskip("torch")
    from dense_gemm_sgemm_gb300 import scaled, update

    for module in (scaled, update):
        for name in module.__all__:
            assert getattr(g, name) is getattr(module, name)
            assert getattr(g, name).__doc__
