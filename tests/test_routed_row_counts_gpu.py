"""Row counts next to 2^31, the documented limit: counters of rows may not wrap there."""
import pytest
import torch

import dense_gemm_sgemm_gb300 as g

pytestmark = pytest.mark.gpu

ROWS = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def room():
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("150 GB of device memory wanted")
    yield
    torch.cuda.empty_cache()


def _off(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rows():
    # 8 columns; ones in the first row and the last few
    x = torch.zeros(ROWS, 8, dtype=torch.float16, device="cuda")
    x[0], x[-40:] = 1.0, 2.0
    return x


def test_no_terms():
    # K = 0 goes to the few-rows kernel whatever the count
    torch.ones(ROWS, 8, dtype=torch.float16, device="cuda")  # what the output's memory held before
    y = g.grouped_linear(torch.empty(ROWS, 0, dtype=torch.float16, device="cuda"),
                         torch.empty(1, 1, 0, dtype=torch.float16, device="cuda"), _off(0, ROWS))
    assert y.shape == (ROWS, 1) and not y[:1000].any() and not y[-10000:].any()


def test_one_group_and_a_short_last_one():
    x, w = _rows(), torch.ones(2, 8, 8, dtype=torch.float16, device="cuda")
    w[1] = 3.0
    for off, last in (((0, ROWS, ROWS), 16.0), ((0, ROWS - 5, ROWS), 48.0)):
        y = g.grouped_linear(x, w, _off(*off))
        assert (y[0] == 8.0).all() and not y[1:5000].any()
        assert not y[-5000:-40].any() and (y[-40:-5] == 16.0).all() and (y[-5:] == last).all()
        del y
    assert g.gemm_get_device_status() == 0
