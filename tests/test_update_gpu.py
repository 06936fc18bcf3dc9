"""The orthogonalised update against its formula in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
QUINTIC = (3.4445, -4.7750, 2.0315)
# The header's figures for what a result is off, relative to its norm, before its own rounding, which adds at most half a
# step of each element: one product of fp16 values (bf16 results, both sides above 128), or three of the parts.
# Three: an error of X grows at most by the polynomial's steepest slope, 3.4445, a step, 485 times over five; the parts hold
# 22 bits and the sums 23 or more, so what a step adds is at most 2^-21 of the norm, and 485 * 2^-21 = 2.3e-4.  (Rank-one
# matrices, whose error has the smallest values to grow from, come to 1e-4; with exact sums it would be 3.4e-5.)
ONE, THREE = 2e-3, 2.5e-4
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def g():
    import dense_gemm_sgemm_gb300 as g

    g.load()
    return g


def formula(m, steps=5, coefficients=QUINTIC, eps=1e-7):
    x = m.double()
    x = x / (x.norm() + eps)
    if m.shape[0] > m.shape[1]:
        x = x.T
    for _ in range(steps):
        a = x @ x.T
        x = coefficients[0] * x + (coefficients[1] * a + coefficients[2] * a @ a) @ x
    return x.T if m.shape[0] > m.shape[1] else x


def near(got, m, wanted=None, dtype=torch.bfloat16, **kw):
    wanted = formula(m, **kw) if wanted is None else wanted
    assert got.dtype == dtype and got.shape == m.shape
    off = (got.double() - wanted).norm() / wanted.norm()
    one = dtype == torch.bfloat16 and min(m.shape) > 128
    assert off <= (ONE if one else THREE) + HALF_STEP[dtype], off


def matrix(rows, cols, kind="normal", seed=0, dtype=torch.float32):
    r = torch.Generator().manual_seed(seed)
    n = min(rows, cols)
    if kind == "normal":
        m = torch.randn(rows, cols, generator=r)
    elif kind == "low":
        rank = max(1, n // 8)
        m = torch.randn(rows, rank, generator=r) @ torch.randn(rank, cols, generator=r) + 0.1 * torch.randn(rows, cols, generator=r)
    elif kind == "one":  # rank one, a few rows and columns dominating
        m = torch.randn(rows, 1, generator=r) ** 5 * torch.randn(1, cols, generator=r) ** 5
    elif kind == "graded":  # singular values over five decades
        u = torch.linalg.qr(torch.randn(rows, n, generator=r)).Q
        v = torch.linalg.qr(torch.randn(cols, n, generator=r)).Q
        m = (u * torch.exp(-torch.linspace(0, 12, n))) @ v.T
    return m.to(dtype).cuda()


SHAPES = [(1, 1), (1, 7), (7, 1), (2, 3), (16, 16), (33, 65), (65, 33), (128, 128), (129, 300), (300, 129), (256, 512), (520, 1000),
          (1000, 520), (640, 640)]


@pytest.mark.parametrize("form", ["", "0", "1", "2", "3"])
@pytest.mark.parametrize("shape", SHAPES)
def test_against_the_formula(g, monkeypatch, shape, form):
    monkeypatch.setenv("GEMM_GB300_ORTHOGONAL_FORM", form)
    for kind in ("normal", "low", "one", "graded"):
        for dtype in (torch.float32, torch.bfloat16) if kind == "normal" else (torch.float32,):
            m = matrix(*shape, kind, dtype=dtype)
            near(g.orthogonalize(m), m)
        for dtype in (torch.float32, torch.float16):
            near(g.orthogonalize(m, out_dtype=dtype), m, dtype=dtype)
    assert g.gemm_get_device_status() == 0


@pytest.mark.parametrize("shape", [(2048, 1024), (1024, 4096), (2500, 2500), (1100, 1300), (1900, 900)])
def test_large_matrices(g, shape):
    for kind in ("normal", "low"):
        m = matrix(*shape, kind)
        near(g.orthogonalize(m), m)
    near(g.orthogonalize(m, out_dtype=torch.float32), m, dtype=torch.float32)


def test_one_step_element_by_element(g):
    # after one step every element is near: half a step of fp16, 2^-11, for each factor of a product (X twice in A, A
    # twice in A^2 beside the sum itself, then B and X: eight at most), and of X's own smallest step, 2^-25 of 2^14
    for shape in ((100, 200), (300, 100)):
        m = matrix(*shape)
        got, wanted = g.orthogonalize(m, steps=1).double(), formula(m, steps=1)
        x = m.double() / m.double().norm()
        x = x.T if shape[0] > shape[1] else x
        a = x.abs() @ x.abs().T
        size = (4.7750 * a + 2.0315 * a @ a) @ x.abs()
        size = size.T if shape[0] > shape[1] else size
        assert ((got - wanted).abs() <= HALF_STEP[torch.bfloat16] * wanted.abs() + 8 * 2.0 ** -11 * size + 1e-9).all()


@pytest.mark.parametrize("form", ["0", "1", "2", "3"])
@pytest.mark.parametrize("shape", [(3, 40, 60), (5, 300, 130), (2, 256, 256), (17, 16, 24)])
def test_stacks(g, monkeypatch, shape, form):
    monkeypatch.setenv("GEMM_GB300_ORTHOGONAL_FORM", form)
    r = torch.Generator().manual_seed(3)
    m = torch.randn(shape, generator=r).cuda() * 10.0 ** torch.arange(shape[0]).reshape(-1, 1, 1).cuda().fmod(7)
    y = g.orthogonalize(m)
    for i in range(shape[0]):
        near(y[i], m[i])
        assert torch.equal(y[i], g.orthogonalize(m[i]))  # the same as alone


def test_other_coefficients_and_steps(g):
    m = matrix(200, 300)
    near(g.orthogonalize(m, steps=12, coefficients=(1.5, -0.5, 0.0)), m, steps=12, coefficients=(1.5, -0.5, 0.0))
    near(g.orthogonalize(m, steps=3, coefficients=(2.0, -1.5, 0.5)), m, steps=3, coefficients=(2.0, -1.5, 0.5))
    each = [(4.0, -6.0, 2.5), (3.0, -4.0, 1.7), (1.875, -1.25, 0.375)]
    x = formula(m, steps=1, coefficients=each[0])
    for c in each[1:]:
        a = x @ x.T
        x = c[0] * x + (c[1] * a + c[2] * a @ a) @ x
    near(g.orthogonalize(m, steps=3, coefficients=each), m, wanted=x)


@pytest.mark.parametrize("scale", [1e-38, 1e-25, 1e-12, 1.0, 1e12, 1e30])
def test_any_magnitude(g, scale):
    m = matrix(96, 160) * scale
    near(g.orthogonalize(m, eps=0.0), m, eps=0.0)
    if scale < 1e-7:
        near(g.orthogonalize(m, eps=scale), m, eps=scale)


def test_norms_across_ranges(g):
    # squares are summed in three ranges, of magnitudes below 2^-40, up to 2^40 and above: matrices with parts of the
    # norm in two of them, and with the ends of fp32
    r = torch.Generator().manual_seed(9)
    sign = torch.randint(0, 2, (96, 160), generator=r).cuda() * 2.0 - 1.0
    for low, high in ((9.0e-13, 9.2e-13), (1.0e12, 1.2e12), (1e-20, 1e-12), (1.0, 1e13), (1e-45, 1e-44), (2.5e38, 3.4e38), (1e-30, 1e30)):
        m = sign * low
        m[::3, ::2] *= high / low if high / low < 3e38 else 1e20
        m = m.clamp(-3.4e38, 3.4e38)
        for eps in (0.0, 1e-7 if low > 1e-15 else 0.0):
            x = m.double() / (m.double().norm() + eps)
            for _ in range(5):
                a = x @ x.T
                x = QUINTIC[0] * x + (QUINTIC[1] * a + QUINTIC[2] * a @ a) @ x
            near(g.orthogonalize(m, eps=eps), m, wanted=x)
    # eps beside the norm, and up to 10^4 times it, in each range
    for scale in (1e-30, 1e-3, 1e20):
        m = matrix(96, 160) * scale
        for ratio in (1e-3, 1.0, 1e4):
            eps = ratio * float(m.double().norm())
            eps = torch.tensor(eps, dtype=torch.float32).item()
            near(g.orthogonalize(m, eps=eps), m, eps=eps)
    # a norm that is not a number: in each range, beside values of the others
    for bad in (float("nan"), float("inf"), -float("inf")):
        for scale in (1e-30, 1.0, 1e20):
            m = matrix(40, 60) * scale
            m[3, 5] = bad
            assert torch.isnan(g.orthogonalize(m)).all()
            m[7, 7] = 1e25
            assert torch.isnan(g.orthogonalize(m)).all()
    assert torch.equal(g.orthogonalize(torch.zeros(9, 9, device="cuda"), eps=3e38), torch.zeros(9, 9, device="cuda").bfloat16())


def test_zeros_infinities_and_strides(g):
    m = torch.randn(4, 70, 90, generator=torch.Generator().manual_seed(1)).cuda()
    m[1] = 0.0
    m[2, 5, 6] = float("inf")
    y = g.orthogonalize(m)
    near(y[0], m[0])
    near(y[3], m[3])
    assert torch.equal(y[1], torch.zeros_like(y[1])) and torch.isnan(y[2]).all()
    assert torch.equal(g.orthogonalize(m[1], eps=0.0), torch.zeros_like(y[1]))
    room = torch.randn(3, 100, 200, generator=torch.Generator().manual_seed(2)).cuda()
    for part in (room[:, 3:80, 1:150], room[0, ::2, 5:66], room[::2, :, 7:8], room[1:2, 4:5]):
        assert torch.equal(g.orthogonalize(part), g.orthogonalize(part.clone()))
        assert torch.equal(g.orthogonalize(part), g.orthogonalize(part.clone()))
    assert g.orthogonalize(room[:0]).shape == (0, 100, 200) and g.orthogonalize(room[0, :0]).shape == (0, 200)
    assert g.orthogonalize(room[0, :, :0]).shape == (100, 0)


def test_repeats_streams_graphs_and_expired_waits(g, monkeypatch):
    m = matrix(300, 500, "low")
    first = g.orthogonalize(m)
    for _ in range(3):
        assert torch.equal(first, g.orthogonalize(m))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = g.orthogonalize(m, stream=s)
    s.synchronize()
    assert torch.equal(first, other)
    held = m.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = g.orthogonalize(held)
    for seed in (5, 6):
        held.copy_(matrix(300, 500, seed=seed))
        graph.replay()
        assert torch.equal(y, g.orthogonalize(held))
    for form in "0123":
        monkeypatch.setenv("GEMM_GB300_ORTHOGONAL_FORM", form)
        monkeypatch.setenv("GEMM_GB300_TEST_INJECT_STALL", "1")
        g.orthogonalize(m, steps=1)
        assert g.gemm_get_device_status() == 5
        monkeypatch.delenv("GEMM_GB300_TEST_INJECT_STALL")
        assert torch.equal(first, g.orthogonalize(m))
        assert g.gemm_get_device_status() == 0


def test_bad_arguments_are_refused(g):
    m = torch.randn(30, 40, device="cuda")
    for bad in (dict(steps=0), dict(steps=65), dict(eps=-1.0), dict(coefficients=(100.0, 100.0, 100.0)),
                dict(coefficients=(float("nan"), 0.0, 0.0)), dict(coefficients=[(1.5, -0.5, 0.0)]), dict(out_dtype=torch.float64)):
        with pytest.raises((ValueError, TypeError, g.GemmError)):
            g.orthogonalize(m, **bad)
    for x in (m[0], m.double(), m.t(), m.cpu(), m[None, None]):
        with pytest.raises((ValueError, TypeError)):
            g.orthogonalize(x)


def test_two_streams_and_two_graphs(g):
    # work space is each call's own: calls that overlap, and graphs that share torch's memory pool
    ms = [matrix(300, 400, seed=s) for s in range(4)]
    wanted = [g.orthogonalize(m) for m in ms]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [g.orthogonalize(ms[i % 4], stream=streams[i % 2]) for i in range(16)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, wanted[i % 4]) for i, y in enumerate(got))
    graphs, outs, pool = [], [], torch.cuda.graph_pool_handle()
    for m in ms[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            outs.append(g.orthogonalize(m))
        graphs.append(graph)
    for _ in range(3):
        for i in (0, 1):
            graphs[i].replay()
            assert torch.equal(outs[i], wanted[i])


def test_gradient_descends_along_the_update(g):
    # the update of a full-rank gradient has singular values near 1, whatever the gradient's were
    m = matrix(300, 200, "graded")
    s = torch.linalg.svdvals(g.orthogonalize(m, steps=12, coefficients=(1.5, -0.5, 0.0), out_dtype=torch.float32).double())
    t = torch.linalg.svdvals(m.double() / m.double().norm())
    for _ in range(12):
        t = 1.5 * t - 0.5 * t ** 3
    # singular values differ by the 2-norm of the error at most; each of 12 steps adds 2^-21 of the norm and grows what
    # the steps before it added by the cubic's slope, 1.5 at most: less than 3 * 1.5^12 * 2^-21
    assert (s - t.sort(descending=True).values).abs().max() <= 3 * 1.5 ** 12 * 2.0 ** -21
