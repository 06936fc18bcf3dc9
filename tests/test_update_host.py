"""Coefficients of the orthogonalised update that need no GPU to be taken or refused."""
import ctypes

import pytest

from dense_gemm_sgemm_gb300 import _lib, build

P = 4096  # a fake, never dereferenced address
OK, UNSUPPORTED = 0, 3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.mark.parametrize("status,each", [
    # iterates that shrink out of what two fp16 parts hold: every singular value is below 2^-20 before the last step
    (UNSUPPORTED, [(0.5, 0.0, 0.0)] * 64), (UNSUPPORTED, [(0.5, 0.0, 0.0)] * 22), (UNSUPPORTED, [(1e-4, 0.0, 0.0)] * 3),
    (UNSUPPORTED, [(0.0, 0.0, 0.0)] * 2), (UNSUPPORTED, [(0.0, 0.01, 0.0)] * 3),
    # results below what the parts of b A + c A^2 hold
    (UNSUPPORTED, [(0.0, 1e-30, 0.0)]), (UNSUPPORTED, [(1e-4, 0.0, 0.0), (0.0, 0.0, 1e-3)]), (OK, [(0.0, 1e-17, 0.0)]), (OK, [(1.0, 1e-30, 0.0)]),
    (OK, [(0.5, 0.0, 0.0)] * 20), (OK, [(1e-4, 0.0, 0.0)] * 2), (OK, [(0.0, 0.0, 0.0)]), (OK, [(0.0, 0.01, 0.0)] * 2),
    (OK, [(1.5, -0.5, 0.0)] * 64), (OK, [(3.4445, -4.7750, 2.0315)] * 64),
])
def test_coefficients(lib, status, each):
    values = (ctypes.c_float * (3 * len(each)))(*[v for c in each for v in c])
    # no matrix: nothing is launched where the coefficients are taken
    assert lib.gemm_orthogonalize(0, 2, 0, 10, 20, P, 20, 200, len(each), values, 1e-7, P, 24, 240, P, None) == status
