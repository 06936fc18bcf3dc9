"""What the orthogonalised update promises of its results: the stated precision for matrices whose elements are alike, whose
roundings are alike too and do not average out, and the same bits in every form and stack."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import dense_gemm_sgemm_gb300 as g

    g.load()
    return g


QUINTIC = (3.4445, -4.7750, 2.0315)


def formula(m):
    x = m.double()
    x = x / (x.norm() + 1e-7)
    x = x.T if m.shape[0] > m.shape[1] else x
    for _ in range(5):
        a = x @ x.T
        x = QUINTIC[0] * x + (QUINTIC[1] * a + QUINTIC[2] * a @ a) @ x
    return x.T if m.shape[0] > m.shape[1] else x


def limit(rows, cols):
    """The header's: 2.5e-4 of the parts and the epilogues, and of the sums, which the longer side adds to.  A sum of K
    products is K / 16 additions in fp32, each off by a step of the sum at most: K / 16 * 2^-23 of it, whatever the
    terms of one sign.  A singular value s whose three sums a step are all off by a relative d, each the way that harms
    most, ends off by at most 98 d over five steps (largest at s = 0.62: of step i its polynomial's terms over its
    value, times the later steps' |s p'(s) / p(s)|)."""
    return 2.5e-4 + 98 * 2.0 ** -23 * max(rows, cols) / 16


def matrix(rows, cols, kind):
    r = torch.Generator().manual_seed(7)
    n, i = min(rows, cols), torch.arange(min(rows, cols))
    if kind == "constant":
        m = torch.full((rows, cols), 0.7)
    elif kind == "ones":
        m = torch.ones(rows, cols)
    elif kind == "signs":  # rank one
        m = torch.where(torch.randn(rows, 1, generator=r) * torch.randn(1, cols, generator=r) > 0, 1.0, -1.0)
        m = m[:, :1] * m[:1]
    elif kind == "equal rows":
        m = torch.randn(1, cols, generator=r).expand(rows, cols)
    elif kind == "four blocks":  # the gradient of a classifier
        m = (torch.arange(rows)[:, None] * 4 // rows == torch.arange(cols) * 4 // cols).float()
    elif kind == "many blocks":
        m = (torch.arange(rows)[:, None] * 32 // rows == torch.arange(cols) * 32 // cols).float()
    elif kind == "pairs":
        m = torch.zeros(rows, cols)
        m[i, i] = m[i, (i ^ 1).clamp(max=n - 1)] = 1.0
    elif kind == "identity":
        m = torch.eye(rows, cols)
    elif kind == "two":  # singular values of which the sums' errors grow most
        m = torch.randn(rows, 1, generator=r) * torch.randn(1, cols, generator=r)
        m += 0.7 * torch.randn(rows, 1, generator=r) * torch.randn(1, cols, generator=r)
    elif kind == "normal":
        m = torch.randn(rows, cols, generator=r)
    return m.contiguous().cuda()


KINDS = ["constant", "ones", "signs", "equal rows", "four blocks", "many blocks", "pairs", "identity", "two", "normal"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", [(129, 129), (129, 300), (256, 256), (256, 512), (512, 512), (520, 1000), (1000, 520), (1024, 1024)])
def test_precision_where_roundings_are_alike(g, shape, kind):
    m = matrix(*shape, kind)
    wanted = formula(m)
    size, most = wanted.norm(), limit(*shape)
    whole = g.orthogonalize(m, out_dtype=torch.float32)
    assert (whole.double() - wanted).norm() / size <= most
    for dtype in (torch.bfloat16, torch.float16):
        got = g.orthogonalize(m, out_dtype=dtype)
        # the one rounding of the same result; beside the formula's own rounding it is off by at most twice what the
        # result is: |round(y) - w| <= |round(y) - y| + |y - w| <= |round(w) - y| + |y - w| <= |round(w) - w| + 2 |y - w|
        assert torch.equal(got, whole.to(dtype))
        rounding = (wanted.to(dtype).double() - wanted).norm() / size
        assert (got.double() - wanted).norm() / size <= rounding + 2 * most


@pytest.mark.parametrize("kind", ["constant", "ones", "equal rows", "four blocks", "two", "normal"])
@pytest.mark.parametrize("shape", [(2048, 4096), (4096, 1500), (4096, 4096)])
def test_precision_of_long_sums(g, shape, kind):
    m = matrix(*shape, kind)
    wanted = formula(m)
    size, most = wanted.norm(), limit(*shape)
    whole = g.orthogonalize(m, out_dtype=torch.float32)
    assert (whole.double() - wanted).norm() / size <= most
    assert torch.equal(g.orthogonalize(m), whole.bfloat16())


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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("each", [[(0.5, 0.0, 0.0)] * 20, [(0.01, 0.0, 0.0)] * 4, [(0.0, -0.03, 0.0), (0.0, 1.0, 0.0)], [(0.0, 0.0, 0.0)],
                                  [(0.02, 0.0, 0.0), (2.0, -1.5, 0.5)], [(0.0, 1e-17, 0.0)], [(0.0, 0.0, -1e-17)]])
def test_steps_that_shrink_the_iterate(g, each, dtype):
    # what an iterate loses is in proportion to its own bound, whatever that is; a step's three products and
    # epilogues are off by less than 2^-20, which no step here grows to more than 9 times (the fifth power's 5, the cube's 3)
    for m in (normal(200, 300), torch.ones(300, 140, device="cuda")):
        x = m.double() / (m.double().norm() + 1e-7)
        for a, b, c in each:
            s = x @ x.T
            x = a * x + (b * s + c * s @ s) @ x
        got = g.orthogonalize(m, steps=len(each), coefficients=each, out_dtype=dtype)
        rounding = (x.to(dtype).double() - x).norm()
        assert (got.double() - x).norm() <= rounding + 2 * len(each) * 9 * 2.0 ** -20 * x.norm()
    with pytest.raises(g.GemmError):
        g.orthogonalize(m, steps=64, coefficients=(0.5, 0.0, 0.0))
