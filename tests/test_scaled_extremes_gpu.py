"""Block-scaled products with every pair of scales across fp32's range, and sums of zero among them."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
MOST = torch.finfo(torch.float32).max
SCALES = [0.0, 2.0 ** -149, 1.5 * 2.0 ** -126, 2.0 ** -64, 2.0 ** -41, 1.0, 1e10, 1.5 * 2.0 ** 63, 2.0 ** 64, 1.75 * 2.0 ** 126,
          2.0 ** 127, MOST, -2.0 ** 127, float("inf"), float("nan")]
SUMS = [(0.0, 0.0), (1.0, -1.0), (2.0 ** -16, 0.0), (1.0, 0.5), (-57344.0, 3.0)]  # two codes of a row of A
CODES = [1.0, 2.0 ** -16, 57344.0]  # of a column of B


@pytest.fixture(scope="module")
def g():
    import dense_gemm_sgemm_gb300 as g

    g.load()
    return g


@pytest.mark.parametrize("b_block", [1, 128])
@pytest.mark.parametrize("plan", ["P", "128:1", "64:2", "32:1", "128:1:s", "32:2:s"])
def test_every_pair_of_scales(g, monkeypatch, plan, b_block):
    monkeypatch.setenv("GEMM_GB300_SCALED_PLAN", plan)
    K = 256  # the second block of K adds zeros of scale 1
    a = torch.zeros(len(SCALES) * len(SUMS), K)
    a[:, :2] = torch.tensor(SUMS).repeat(len(SCALES), 1)
    sa = torch.ones(len(a), 2)
    sa[:, 0] = torch.tensor(SCALES).repeat_interleave(len(SUMS))
    for which in [SCALES] if b_block == 1 else [[s] for s in SCALES]:
        b = torch.zeros(len(which) * len(CODES), K)
        b[:, :2] = torch.tensor(CODES).repeat(len(which))[:, None]
        each = torch.tensor(which).repeat_interleave(len(CODES))
        sb = torch.ones(len(b) if b_block == 1 else 1, 2)
        sb[:, 0] = each if b_block == 1 else each[0]
        c = g.scaled_matmul(a.to(torch.float8_e5m2).cuda(), sa.cuda(), b.to(torch.float8_e5m2).cuda(), sb.cuda(), out_dtype=torch.float32)
        # exact in 64 bits; in fp32 the sum, the product of the scales' parts and that of both are rounded: 3 half steps
        wanted = sa[:, :1].double() * each.double() * (a.double() @ b.double().T)
        c = c.cpu()
        assert torch.equal(torch.isnan(c), torch.isnan(wanted))
        beyond = wanted.abs() > MOST * (1 + 2.0 ** -22)
        assert torch.equal(c[beyond], wanted[beyond].float())
        near = wanted.abs() <= MOST * (1 - 2.0 ** -22)
        assert ((c.double() - wanted).abs()[near] <= 3 * 2.0 ** -24 * wanted.abs()[near] + 2.0 ** -149).all()
    assert g.gemm_get_device_status() == 0


def test_reading_back_takes_one_scale_for_a_block(g):
    r = torch.Generator().manual_seed(3)
    for rows, cols in ((2, 2), (5, 300), (300, 2)):  # one for every element
        q = g.quantize_blocks(torch.randn(rows, cols, generator=r).cuda())[0]
        with pytest.raises(ValueError, match="every element"):
            g.dequantize_blocks(q, torch.ones(rows, cols, device="cuda"))
    for rows, cols in ((1, 1), (1, 300), (300, 1)):  # of a single row or column: those of blocks across it
        q = g.quantize_blocks(torch.randn(rows, cols, generator=r).cuda())[0]
        s = torch.rand(rows, cols, generator=r).cuda()
        assert torch.equal(g.dequantize_blocks(q, s, out_dtype=torch.float32), q.float() * s)


def test_chained_calls_read_what_the_call_before_wrote(g):
    # every call takes its place on the SMs while the one before still runs, and writes to memory read a few calls ago
    def chain(x, wait):
        for i in range(60):
            block = ((1, 128), (128, 1), (128, 128))[i % 3]
            q, s = g.quantize_blocks(x, block, dtype=(torch.float8_e4m3fn, torch.float8_e5m2)[i % 2])
            wait()
            x = g.dequantize_blocks(q, s, out_dtype=torch.float32)
            wait()
            x = g.orthogonalize(x, steps=1, coefficients=(-0.9, 0.1, 0.0), out_dtype=torch.float32)
            wait()
        return x

    for shape in ((130, 300), (500, 260)):
        x = torch.randn(shape, generator=torch.Generator().manual_seed(5)).cuda()
        assert torch.equal(chain(x, lambda: None), chain(x, torch.cuda.synchronize))
