"""The routed products' Python binding and its place in the package and the build, without a GPU."""
import pytest

from dense_gemm_sgemm_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_operands_of_two_devices_are_refused():
    # every tensor of a call passes this comparison before anything is allocated or launched
    torch = pytest.importorskip("torch")
    from dense_gemm_sgemm_gb300 import routed

    same = routed._routed.same_device
    same(torch.device("cuda:0"), torch.device("cuda:0"))
    same(torch.device("cuda:1"), torch.device("cuda:1"))
    with pytest.raises(ValueError, match="cuda:1"):
        same(torch.device("cuda:0"), torch.device("cuda:1"))
    with pytest.raises(TypeError):
        same("cuda:0", torch.device("cuda:0"))
