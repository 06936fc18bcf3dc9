"""Block-scaled 8-bit values and products against their plain forms in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

from tests import scaled_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
BLOCKS = [(1, 128), (128, 1), (128, 128)]


@pytest.fixture(scope="module")
def g():
    import dense_gemm_sgemm_gb300 as g

    g.load()
    return g


def gen(seed=0):
    return torch.Generator().manual_seed(seed)


def same_codes(q, scales, x, block, dtype):
    codes, wanted = ref.quantise(x, block, dtype)
    assert q.dtype == dtype and q.shape == x.shape
    assert torch.equal(scales.cpu(), wanted)
    got = q.view(torch.uint8).cpu() if q.is_contiguous() else q.cpu().contiguous().view(torch.uint8)
    nan = (codes & 0x7F) == 0x7F if dtype == E4 else (codes & 0x7F) > 0x7C
    assert torch.equal(torch.where(nan, codes & 0x7F, codes), torch.where(nan, got & 0x7F, got))


def spread(rows, cols, dtype, seed=0):
    """Values over many powers of two, zeros and blocks of zeros among them."""
    r = gen(seed)
    x = torch.randn(rows, cols, generator=r) * 2.0 ** torch.randint(-12, 13, (rows, cols), generator=r)
    x[torch.rand(rows, cols, generator=r) < 0.1] = 0.0
    x[:, 128:256] = 0.0
    x[rows // 2:rows // 2 + 2] *= 2.0 ** -14
    return x.clamp(-60000, 60000).to(dtype)


# ------------------------------------------------------------------ quantising
@pytest.mark.parametrize("shape", [(1, 1), (1, 128), (1, 300), (2, 16), (3, 129), (127, 7), (128, 128), (129, 257), (300, 1000), (2000, 384)])
@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("dtype", [E4, E5])
def test_quantise(g, shape, block, dtype):
    for t in (torch.float32, torch.float16, torch.bfloat16):
        x = spread(*shape, t)
        q, s = g.quantize_blocks(x.cuda(), block, dtype=dtype)
        same_codes(q, s, x, block, dtype)


@pytest.mark.parametrize("shape", [(1, 1), (5, 200), (128, 128), (333, 1040), (4000, 136)])
def test_quantise_both(g, shape):
    x = spread(*shape, torch.bfloat16)
    q, s, qc, sc = g.quantize_both(x.cuda(), dtype=E5)
    same_codes(q, s, x, (1, 128), E5)
    same_codes(qc, sc, x, (128, 1), E5)


@pytest.mark.parametrize("dtype", [E4, E5])
def test_every_binade_and_border(g, dtype):
    # maxima from fp32's smallest to its largest, one to a row, beside every ratio of nine bits
    e = torch.arange(-149, 128)
    m = 1 + torch.arange(256).float() / 256
    x = (m[None, :].double() * 2.0 ** e[:, None].double()).float()
    x[:, 128:] *= -1
    q, s = g.quantize_blocks(x.cuda(), dtype=dtype)
    same_codes(q, s, x, (1, 128), dtype)
    assert torch.isfinite(ref.values(q.cpu(), s.cpu())).all()


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("dtype", [E4, E5])
def test_non_finite_values_stay_alone(g, block, dtype):
    x = spread(200, 300, torch.float32)
    for i, v in enumerate((float("inf"), float("-inf"), float("nan"))):
        x[7 + 50 * i, 5 + 90 * i] = v
    q, s = g.quantize_blocks(x.cuda(), block, dtype=dtype)
    same_codes(q, s, x, block, dtype)
    assert torch.isnan(q.float()).sum() == 3


@pytest.mark.parametrize("dtype", [E4, E5])
@pytest.mark.parametrize("t", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("shape", [(256, 384), (200, 300), (16, 256), (2050, 264)])
def test_non_finite_and_tiny_values_of_every_type(g, shape, t, dtype):
    # both ways at once: infinities and NaN in whole pieces, rows, columns and blocks, and values down to the type's least
    r = gen(33)
    x = torch.randn(shape, generator=r) * 2.0 ** torch.randint(-12, 13, shape, generator=r)
    least = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}[t]
    x[:, 16:24] = least * torch.randint(-3, 4, (shape[0], 8), generator=r)
    x[9] = least * torch.randint(0, 3, (shape[1],), generator=r)
    x[5, :] = float("nan")
    x[11, 8:16] = float("inf")
    x[3, 40:48] = torch.tensor([float("nan"), -float("inf")]).repeat(4)
    x[:, 130] = -float("inf")
    x[:, 131] = float("nan")
    if shape[0] >= 256:
        x[128:256, 128:256] = float("nan")
    x[torch.rand(shape, generator=r) < 0.01] = float("nan")
    x = x.clamp(-65504, 65504).to(t) if t == torch.float16 else x.to(t)
    x[2, 3], x[2, 200] = float("inf"), -float("inf")
    q, s, qc, sc = g.quantize_both(x.cuda(), dtype=dtype)
    same_codes(q, s, x, (1, 128), dtype)
    same_codes(qc, sc, x, (128, 1), dtype)
    for block in BLOCKS:
        same_codes(*g.quantize_blocks(x.cuda(), block, dtype=dtype), x, block, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_any_stride_and_alignment(g, dtype):
    room = torch.randn(400, 333, generator=gen()).to(dtype).cuda()
    for x in (room[:, 1:], room[3:, :129], room[::2, 5:300], room[7:8, 3:], room.new_zeros(0, 64), room.new_zeros(5, 0)):
        for block in BLOCKS:
            q, s = g.quantize_blocks(x, block)
            assert s.shape == (-(-x.shape[0] // block[0]), -(-x.shape[1] // block[1]))
            if x.numel():
                same_codes(q, s, x, block, E4)


@pytest.mark.parametrize("shape", [(1, 1), (1, 40), (40, 1), (130, 17), (300, 1000)])
@pytest.mark.parametrize("dtype", [E4, E5])
def test_read_back(g, shape, dtype):
    x = spread(*shape, torch.bfloat16)
    for block in BLOCKS:
        q, s = g.quantize_blocks(x.cuda(), block, dtype=dtype)
        for t in (torch.float32, torch.float16, torch.bfloat16):
            wanted = ref.values(q.cpu(), s.cpu()).float().to(t)
            assert torch.equal(g.dequantize_blocks(q, s, out_dtype=t).cpu(), wanted)
    s = torch.rand(s.shape, generator=gen())  # any scales
    wanted = ref.values(q.cpu(), s).to(torch.float32)
    assert torch.equal(g.dequantize_blocks(q, s.cuda(), out_dtype=torch.float32).cpu(), wanted)


# ------------------------------------------------------------------ products
PLANS = ["", "P", "128:1", "128:2", "64:1", "64:4", "32:8", "32:1", "128:4:s", "64:2:s", "32:1:s"]


def on_gpu(*tensors):
    return [ref.stored(t.cuda()) if t.dtype in (E4, E5) else t.cuda() for t in tensors]


def run(g, a, sa, b, sb, **kw):
    return g.scaled_matmul(*on_gpu(a, sa, b, sb), **kw)


@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("ops", ["NT", "NN", "TT", "TN"])
def test_whole_numbers_are_exact(g, monkeypatch, plan, ops):
    monkeypatch.setenv("GEMM_GB300_SCALED_PLAN", plan)
    r = gen(1)
    for M, N, K, ablk, bblk, ta, tb in [(1, 1, 1, 1, 128, E4, E4), (5, 300, 1100, 1, 128, E4, E4), (300, 260, 640, 1, 1, E5, E4),
                                        (129, 65, 257, 128, 1, E4, E5), (520, 513, 1024, 1, 128, E5, E5), (64, 32, 2048, 128, 128, E4, E4)]:
        a, sa = ref.operand(r, M, K, ops[0] == "T", ablk, ta)
        b, sb = ref.operand(r, N, K, ops[1] == "N", bblk, tb)
        wanted, _ = ref.product(a, sa, b, sb, ops[0], ops[1])
        for t in (torch.float32, torch.bfloat16):
            c = run(g, a, sa, b, sb, opA=ops[0], opB=ops[1], out_dtype=t)
            assert torch.equal(c.cpu(), wanted.to(t)), (M, N, K, ablk, bblk, t)
    assert g.gemm_get_device_status() == 0


@pytest.mark.parametrize("plan", ["", "P", "128:1", "64:2:s", "32:4"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_any_values(g, monkeypatch, plan, dtype):
    monkeypatch.setenv("GEMM_GB300_SCALED_PLAN", plan)
    r = gen(2)
    for M, N, K, bblk in [(1, 2304, 1000, 128), (33, 500, 4096, 128), (1001, 777, 513, 128), (400, 300, 2500, 1)]:
        a, sa = ref.operand(r, M, K, False, 1, E4, ints=False)
        b, sb = ref.operand(r, N, K, False, bblk, E4, ints=False)
        wanted, bound = ref.product(a, sa * 1e-3, b, sb * 1e-3, dtype=dtype)
        c = run(g, a, sa * 1e-3, b, sb * 1e-3, out_dtype=dtype).cpu().double()
        off = (c - wanted).abs()
        assert (off <= bound).all(), (M, N, K, (off / bound).max())


def test_large_problem_with_several_tiles_a_pair(g):
    r = gen(3)
    a, sa = ref.operand(r, 4100, 384, False, 1, E4)
    b, sb = ref.operand(r, 2900, 384, False, 128, E4)
    wanted, _ = ref.product(a.cuda(), sa.cuda(), b.cuda(), sb.cuda())
    for t in (torch.float32, torch.float16):
        assert torch.equal(run(g, a, sa, b, sb, out_dtype=t), wanted.to(t))
    sb = torch.repeat_interleave(sb, 128, 0)[:2900]
    assert torch.equal(run(g, a, sa, b, sb, out_dtype=torch.float32), wanted.float())


@pytest.mark.parametrize("splits", [1, 2, 8])
@pytest.mark.parametrize("ops", ["NT", "NN", "TN"])
def test_tiles_beyond_the_last_full_wave(g, monkeypatch, splits, ops):
    monkeypatch.setenv("GEMM_GB300_SCALED_PLAN", f"P:{splits}")
    r = gen(31)
    for M, N, bblk in [(2500, 2200, 128), (2050, 2580, 1)]:  # 90 and 99 tiles, quarters of some outside the matrix
        a, sa = ref.operand(r, M, 1100, ops[0] == "T", 1, E4)
        b, sb = ref.operand(r, N, 1100, ops[1] == "N", bblk, E4)
        wanted, _ = ref.product(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), ops[0], ops[1])
        for t in (torch.float32, torch.bfloat16):
            assert torch.equal(run(g, a, sa, b, sb, opA=ops[0], opB=ops[1], out_dtype=t), wanted.to(t)), (M, N, t)
    assert g.gemm_get_device_status() == 0


def test_tail_of_single_tiles_in_a_chain(g, monkeypatch):
    # what is right ahead of and behind the two kernels, over the same memory, eagerly and replayed
    monkeypatch.setenv("GEMM_GB300_SCALED_PLAN", "P:2")
    r = gen(32)
    x = torch.randn(2500, 2304, generator=r).bfloat16().cuda()
    q, s = g.quantize_blocks(torch.randn(2200, 2304, generator=r).cuda(), (128, 128))

    def chain():
        y = x
        for _ in range(3):
            y = g.scaled_matmul(*g.quantize_blocks(y), *((q, s) if y is x else (q2, s2)))
        return y

    q2, s2 = g.quantize_blocks(torch.randn(2200, 2200, generator=r).cuda(), (128, 128))
    torch.cuda.synchronize()
    wanted = x
    for w in ((q, s), (q2, s2), (q2, s2)):
        xq = g.quantize_blocks(wanted)
        torch.cuda.synchronize()
        wanted = g.scaled_matmul(*xq, *w)
        torch.cuda.synchronize()
    for _ in range(5):
        assert torch.equal(chain(), wanted)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = chain()
    for _ in range(5):
        y.zero_()
        graph.replay()
        assert torch.equal(y, wanted)


def test_tails_of_two_streams_at_once(g, monkeypatch):
    monkeypatch.setenv("GEMM_GB300_SCALED_PLAN", "P:4")
    r = gen(34)
    w = g.quantize_blocks(torch.randn(2300, 1536, generator=r).cuda(), (128, 128))
    xs = [torch.randn(2304, 1536, generator=r).bfloat16().cuda() for _ in range(2)]
    wanted = [g.quantize_blocks(g.scaled_matmul(*g.quantize_blocks(x), *w)) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(15):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(g.quantize_blocks(g.scaled_matmul(*g.quantize_blocks(xs[i]), *w)))
    torch.cuda.synchronize()
    for i in range(2):
        for q, s in got[i]:
            assert torch.equal(q.view(torch.uint8), wanted[i][0].view(torch.uint8)) and torch.equal(s, wanted[i][1])
    assert g.gemm_get_device_status() == 0


@pytest.mark.parametrize("plan", ["P", "128:2", "32:1:s"])
@pytest.mark.parametrize("bblk", [1, 128])
def test_scales_of_any_size(g, monkeypatch, plan, bblk):
    # products of scales below and beyond fp32's range, whose results fp32 holds; zero scales of either sign of zero
    monkeypatch.setenv("GEMM_GB300_SCALED_PLAN", plan)
    r = gen(4)
    M, N, K = 20, 30, 512
    a, sa = ref.operand(r, M, K, False, 1, E4)
    b, sb = ref.operand(r, N, K, False, bblk, E4)
    for pa, pb in [(-120, 118), (100, -126), (126, -120), (-126, 20), (-70, -70), (70, 50), (-149, 140), (60, -60)]:
        x, y = sa * 2.0 ** pa, sb * 2.0 ** pb
        x[3] = 0.0
        x[:, 1] *= 0.5
        if not (torch.isfinite(x).all() and torch.isfinite(y).all()):
            x, y = x.clamp(max=2.0 ** 127), y.clamp(max=2.0 ** 127)
        wanted, bound = ref.product(a, x, b, y)
        c = run(g, a, x, b, y, out_dtype=torch.float32).cpu()
        # any partial sum is at most the sum of the magnitudes: below fp32's largest value, 3.4e38, none overflows
        # (where one does, the rest of the row may be of the other sign and the result infinite though it would fit)
        fits = ref.values(a, x).abs() @ ref.values(b, y).abs().T < 3e38
        assert ((c.double() - wanted).abs() <= bound + 2.0 ** -147)[fits].all(), (pa, pb)
        # beyond it no finite result is right; two partial sums may be infinite with opposite signs
        assert not torch.isfinite(c[wanted.abs() > 3.5e38]).any()


@pytest.mark.parametrize("plan", ["P", "128:1", "64:2:s", "32:2"])
def test_nan_codes_and_scales_stay_in_their_rows(g, monkeypatch, plan):
    monkeypatch.setenv("GEMM_GB300_SCALED_PLAN", plan)
    r = gen(5)
    a, sa = ref.operand(r, 140, 700, False, 1, E4)
    b, sb = ref.operand(r, 150, 700, False, 1, E4)
    wanted, _ = ref.product(a, sa, b, sb)
    a.view(torch.uint8)[17, 699] = 0x7F
    sa = sa.clone()
    sa[90, 2] = float("nan")
    sb = sb.clone()
    sb[40, 5] = float("nan")
    c = run(g, a, sa, b, sb, out_dtype=torch.float32).cpu()
    hit = torch.zeros_like(c, dtype=torch.bool)
    hit[17], hit[90], hit[:, 40] = True, True, True
    assert torch.isnan(c[hit]).all() and torch.equal(c[~hit], wanted.float()[~hit])


def test_strides_of_operands_and_scales(g):
    r = gen(6)
    M, N, K = 100, 90, 300
    a, sa = ref.operand(r, M, K, False, 1, E4)
    b, sb = ref.operand(r, N, K, False, 128, E4)
    wanted, _ = ref.product(a, sa, b, sb, dtype=torch.float32)
    room = torch.zeros(M, 640, dtype=torch.uint8, device="cuda").view(E4)
    wide = room[:, 32:32 + K]
    wide.copy_(a)
    spaced = torch.zeros(2 * M, 7, device="cuda")[::2, 1:4]
    spaced.copy_(sa)
    one = sb[:, :1].contiguous().expand(sb.shape).cuda()  # stride 0
    b1, sb1 = b, sb[:, :1].expand(sb.shape).contiguous()
    assert torch.equal(g.scaled_matmul(wide, spaced, *on_gpu(b, sb), out_dtype=torch.float32).cpu(), wanted.float())
    wanted, _ = ref.product(a, sa, b1, sb1)
    assert torch.equal(g.scaled_matmul(wide, spaced, *on_gpu(b), one, out_dtype=torch.float32).cpu(), wanted.float())


def test_empty_sizes(g):
    z = torch.zeros(0, 256, dtype=torch.uint8, device="cuda").view(E4)
    w = torch.zeros(64, 256, dtype=torch.uint8, device="cuda").view(E4)
    s, ws = torch.zeros(0, 2, device="cuda"), torch.ones(1, 2, device="cuda")
    assert g.scaled_matmul(z, s, w, ws).shape == (0, 64)
    assert g.scaled_matmul(w, ws, z, s).shape == (64, 0)
    e = torch.zeros(5, 0, dtype=torch.uint8, device="cuda").view(E4)
    c = g.scaled_matmul(e, torch.zeros(5, 0, device="cuda"), e, torch.zeros(5, 0, device="cuda"))
    assert torch.equal(c, torch.zeros(5, 5, device="cuda", dtype=torch.bfloat16))


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (77, 1000, 2000), (2048, 2048, 512)])
def test_same_bits_every_time_and_in_a_graph(g, M, N, K):
    r = gen(7)
    a, sa = on_gpu(*ref.operand(r, M, K, False, 1, E4, ints=False))
    b, sb = on_gpu(*ref.operand(r, N, K, False, 128, E4, ints=False))
    first = g.scaled_matmul(a, sa, b, sb)
    for _ in range(5):
        assert torch.equal(first, g.scaled_matmul(a, sa, b, sb))
    x = torch.randn(M, K, generator=r).cuda()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        q, s = g.quantize_blocks(x)
        y = g.scaled_matmul(q, s, b, sb)
    for _ in range(3):
        x.copy_(torch.randn(M, K, generator=r))
        graph.replay()
        q1, s1 = g.quantize_blocks(x)
        assert torch.equal(y, g.scaled_matmul(q1, s1, b, sb))


def test_layer_of_8_bit_products(g):
    # forward, input and weight gradients in a run, each against the values that were really quantised
    r = gen(8)
    T, N, K = 333, 520, 1040
    x, w, dy = torch.randn(T, K, generator=r), torch.randn(N, K, generator=r) / 32, torch.randn(T, N, generator=r) * 1e-3
    wq, ws = g.quantize_blocks(w.cuda(), (128, 128))
    xq, xs, xc, xcs = g.quantize_both(x.bfloat16().cuda())
    y = g.scaled_matmul(xq, xs, wq, ws)
    dq, ds, dc, dcs = g.quantize_both(dy.bfloat16().cuda(), dtype=E5)
    dx = g.scaled_matmul(dq, ds, wq, ws, opB="N")
    dw = g.scaled_matmul(dc, dcs, xc, xcs, opA="T", opB="N", out_dtype=torch.float32)
    for c, args, ops, t in [(y, (xq, xs, wq, ws), "NT", torch.bfloat16), (dx, (dq, ds, wq, ws), "NN", torch.bfloat16),
                            (dw, (dc, dcs, xc, xcs), "TN", torch.float32)]:
        wanted, bound = ref.product(*(v.cpu() for v in args), *ops, dtype=t)
        assert ((c.cpu().double() - wanted).abs() <= bound).all()
    # quantising costs each factor half a step: 2^-4 of e4m3's values, 2^-3 of e5m2's, and below the smallest normal
    # value half of e4m3's smallest step, s 2^-10 with s <= max 2 / 448: as 2^-4 of at most max 2^-13
    for c, p, q, off in [(y, x.bfloat16(), w.T, 2 * 2.0 ** -4 + 2.0 ** -8), (dw, dy.bfloat16().T, x.bfloat16(), 2.0 ** -3 + 2.0 ** -4 + 2.0 ** -7)]:
        p, q = p.double(), q.double()
        size = (p.abs() + p.abs().max() * 2.0 ** -13) @ (q.abs() + q.abs().max() * 2.0 ** -13)
        assert ((c.cpu().double() - p @ q).abs() <= 1.01 * off * size).all()


def test_other_streams_and_expired_waits(g, monkeypatch):
    r = gen(9)
    a, sa = on_gpu(*ref.operand(r, 300, 512, False, 1, E4))
    b, sb = on_gpu(*ref.operand(r, 512, 512, False, 128, E4))
    torch.cuda.synchronize()
    wanted = g.scaled_matmul(a, sa, b, sb)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = g.scaled_matmul(a, sa, b, sb, stream=s)
    s.synchronize()
    assert torch.equal(got, wanted)
    for plan in ("P", "128:1", "64:4:s"):
        monkeypatch.setenv("GEMM_GB300_SCALED_PLAN", plan)
        monkeypatch.setenv("GEMM_GB300_TEST_INJECT_STALL", "1")
        g.scaled_matmul(a, sa, b, sb)
        assert g.gemm_get_device_status() == 5
        monkeypatch.delenv("GEMM_GB300_TEST_INJECT_STALL")
        assert torch.equal(g.scaled_matmul(a, sa, b, sb), wanted)
        assert g.gemm_get_device_status() == 0


@pytest.mark.parametrize("bad", [
    lambda q, s, w, ws: (q[:, :200], s, w, ws),                       # inner dimensions differ
    lambda q, s, w, ws: (q, s[:, :1], w, ws),                         # too few scales
    lambda q, s, w, ws: (q, s.half(), w, ws),                         # scales of another type
    lambda q, s, w, ws: (q, s[:, 0], w, ws),                          # not 2-D
    lambda q, s, w, ws: (q, s.repeat_interleave(128, 1)[:, :256], w, ws),  # one for every element
    lambda q, s, w, ws: (q.float(), s, w, ws),                        # not 8-bit
    lambda q, s, w, ws: (q, s, w.t(), ws.t()),                        # column stride
    lambda q, s, w, ws: (q, s.cpu(), w, ws),                          # another device
])
def test_bad_arguments_are_refused(g, bad):
    q, s = g.quantize_blocks(torch.randn(40, 256, device="cuda"))
    w, ws = g.quantize_blocks(torch.randn(200, 256, device="cuda"), (128, 128))
    with pytest.raises((ValueError, TypeError)):
        g.scaled_matmul(*bad(q, s, w, ws))
    with pytest.raises((ValueError, TypeError)):
        g.scaled_matmul(q, s, w, ws, out_dtype=torch.float64)
    with pytest.raises(g.GemmError, match="MISALIGNED"):  # rows off 16-byte boundaries
        g.scaled_matmul(q[:, 8:], s, w[:, 8:], ws)


def test_many_calls_at_once(g):
    # on two streams, plans of every form, through memory that the calls before have used
    r = gen(11)
    cases = []
    for M, N, K, block in [(1, 700, 900, 128), (64, 1500, 1100, 128), (700, 800, 600, 1), (1500, 1300, 300, 128), (2600, 2200, 260, 128)]:
        a, sa = ref.operand(r, M, K, False, 1, E4)
        b, sb = ref.operand(r, N, K, False, block, E4)
        cases.append((on_gpu(a, sa, b, sb), ref.product(a, sa, b, sb)[0].float().cuda()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(60):
        operands, wanted = cases[i * 7 % 5]
        got.append((g.scaled_matmul(*operands, out_dtype=torch.float32, stream=streams[i % 2]), wanted))
    torch.cuda.synchronize()
    assert all(torch.equal(c, wanted) for c, wanted in got)
    assert g.gemm_get_device_status() == 0


def test_offsets_past_32_bits(g):
    # rows whose elements lie more than 2^31 (and bytes more than 2^32) behind the first
    rows, cols = 70000, 32768
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, 10000):
        x[i:i + 10000] = torch.randn(min(10000, rows - i), cols, device="cuda").bfloat16()
    q, s = g.quantize_blocks(x)
    last = slice(rows - 130, rows)
    same_codes(q[last], s[last], x[last].cpu(), (1, 128), E4)
    back = g.dequantize_blocks(q, s)
    assert torch.equal(back[last].cpu(), ref.values(q[last].cpu(), s[last].cpu()).bfloat16())
    del back
    w, ws = g.quantize_blocks(torch.randn(40, cols, device="cuda") / 181, (128, 128))
    y = g.scaled_matmul(q, s, w, ws, out_dtype=torch.float32)
    wanted, bound = ref.product(q[last], s[last].contiguous(), w, ws)
    assert ((y[last].double() - wanted).abs() <= bound).all()
    del y, q, s
    # more than 2^31 results
    a, sa = g.quantize_blocks(torch.ones(66000, 128, device="cuda"))
    c = g.scaled_matmul(a, sa, a, sa)
    assert bool((c[65900:] == 128).all()) and bool((c[:100] == 128).all())
