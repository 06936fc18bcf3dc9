"""What the orthogonalised update promises of its results: the same bits in every form and stack."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import dense_gemm_sgemm_gb300 as g

    g.load()
    return g


def normal(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(129, 129), (140, 300), (255, 400), (256, 256), (300, 500), (520, 1000), (1000, 520), (700, 641)])
def test_every_form_gives_the_same_bits(g, monkeypatch, shape, dtype):
    m = normal(*shape)
    results = []
    for form in ("0", "1", "2", "3", "02", "20", "13", "31"):
        monkeypatch.setenv("GEMM_GB300_ORTHOGONAL_FORM", form)
        results.append(g.orthogonalize(m, out_dtype=dtype))
    assert all(torch.equal(results[0], y) for y in results[1:])
    assert g.gemm_get_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(5, 700, 1300), (9, 700, 1300), (5, 1024, 1024)])
def test_a_matrix_of_a_stack_is_the_same_as_alone(g, shape, dtype):
    # forms as the library chooses them: other ones for the stack than for one matrix
    m = normal(*shape)
    y = g.orthogonalize(m, out_dtype=dtype)
    for i in (0, 1, shape[0] - 1):
        assert torch.equal(y[i], g.orthogonalize(m[i], out_dtype=dtype))
