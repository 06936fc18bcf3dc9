"""The experts' products, their row movement and gradients against plain 64-bit forms."""
import math

import pytest
import torch

import dense_gemm_sgemm_gb300 as g
from tests import routed_reference as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16]


def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen).to(dtype)


def _offsets(counts):
    return torch.cat([torch.zeros(1, dtype=torch.long), torch.tensor(counts).cumsum(0)]).int()


def _padded(x, extra, fill=math.nan):
    """The same values with `extra` columns of NaN behind each row."""
    wide = torch.full((*x.shape[:-1], x.shape[-1] + extra), fill, dtype=x.dtype)
    wide[..., :x.shape[-1]] = x
    return wide.cuda()[..., :x.shape[-1]]


def _pad8(n):
    return (-n) % 8


# rows of each group: none, one, around the kernels' tiles, all in one
COUNTS = [[1], [0, 3, 0, 1], [8, 9, 7, 0, 16], [33, 0, 64, 1, 31], [129, 2, 0, 255, 64], [300, 17], [0, 0]]


def _run(counts, N, K, dtype, opW="T", gather=False, out_dtype=None, seed=0, pad=0, tail=0):
    gen = torch.Generator().manual_seed(seed)
    E, P = len(counts), sum(counts) + tail
    w_shape = (E, N, K) if opW == "T" else (E, K, N)
    w = _randn(gen, *w_shape, dtype=dtype)
    rows = None
    x_rows = P
    if gather:
        x_rows = max(1, P // 3)
        rows = torch.randint(0, x_rows, (P,), generator=gen).int()
    x = _randn(gen, x_rows, K, dtype=dtype)
    off = _offsets(counts)
    y = g.grouped_linear(_padded(x, _pad8(K) + pad), _padded(w, _pad8(w_shape[2]) + pad), off.cuda(),
                         rows=None if rows is None else rows.cuda(), opW=opW, out_dtype=out_dtype)
    assert g.gemm_get_device_status() == 0
    want, size = ref.grouped(x, w, off, rows, opW)
    n = sum(counts)
    ref.assert_within(y[:n], want[:n], ref.sum_bound(K) * size[:n], f"{counts} {N} {K} {opW}")


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("opW", ["T", "N"])
@pytest.mark.parametrize("dtype", TYPES)
def test_groups(counts, opW, dtype):
    _run(counts, 200, 136, dtype, opW, seed=len(counts))


@pytest.mark.parametrize("N,K", [(1, 1), (8, 8), (7, 65), (257, 33), (128, 64), (520, 1000), (96, 2056)])
@pytest.mark.parametrize("opW", ["T", "N"])
def test_odd_sizes(N, K, opW):
    _run([5, 0, 40, 1], N, K, torch.bfloat16, opW, gather=True, out_dtype=torch.float32, seed=N)
    _run([150, 260], N, K, torch.float16, opW, seed=K)


@pytest.mark.parametrize("opW", ["T", "N"])
def test_padded_rows_and_unused_positions(opW):
    # NaN behind every row and in the rows that belong to no group
    _run([3, 70, 0, 200], 104, 72, torch.bfloat16, opW, pad=16, tail=9)
    _run([3, 7, 0, 2], 104, 72, torch.bfloat16, opW, pad=16, tail=9)


@pytest.mark.parametrize("opW", ["T", "N"])
@pytest.mark.parametrize("counts", [[4, 2], [140, 90]])
def test_rows_outside_are_zeros(opW, counts):
    gen = torch.Generator().manual_seed(4)
    P = sum(counts)
    x = _randn(gen, 20, 64, dtype=torch.float16)
    w = _randn(gen, 2, 48, 64, dtype=torch.float16) if opW == "T" else _randn(gen, 2, 64, 48, dtype=torch.float16)
    rows = torch.randint(-3, 24, (P,), generator=gen).int()
    rows[0], rows[1] = -1, 2 ** 31 - 1
    off = _offsets(counts)
    y = g.grouped_linear(x.cuda(), w.cuda(), off.cuda(), rows=rows.cuda(), opW=opW)
    want, size = ref.grouped(x, w, off, rows, opW)
    ref.assert_within(y, want, ref.sum_bound(64) * size)
    assert (y[0] == 0).all() and (y[1] == 0).all()


@pytest.mark.parametrize("counts", [[6, 0, 3], [150, 40, 300]])
def test_other_groups_infinities_stay_there(counts):
    # a row of infinities and NaN reaches its own output row only, though tiles overlap the groups
    gen = torch.Generator().manual_seed(6)
    P, off = sum(counts), _offsets(counts)
    x = _randn(gen, P, 72, dtype=torch.bfloat16)
    bad = [0, counts[0] - 1, P - 1]
    dirty = x.clone()
    dirty[bad] = math.nan
    dirty[bad[0], ::2] = math.inf
    for opW in "TN":
        w = _randn(gen, len(counts), 72, 72, dtype=torch.bfloat16)
        want = g.grouped_linear(x.cuda(), w.cuda(), off.cuda(), opW=opW)
        got = g.grouped_linear(dirty.cuda(), w.cuda(), off.cuda(), opW=opW)
        keep = torch.ones(P, dtype=torch.bool)
        keep[bad] = False
        assert torch.equal(got[keep.cuda()], want[keep.cuda()])
        assert torch.isnan(got[~keep.cuda()]).any(1).all()


@pytest.mark.parametrize("counts", [[1, 0, 5], [20, 33], [160, 0, 290]])
@pytest.mark.parametrize("I,K", [(24, 64), (129, 200), (72, 1032)])
@pytest.mark.parametrize("dtype", TYPES)
def test_gated(counts, I, K, dtype):
    gen = torch.Generator().manual_seed(I)
    P = sum(counts)
    x = _randn(gen, P, K, dtype=dtype)
    w = (_randn(gen, len(counts), 2 * I, K) * K ** -0.5).to(dtype)
    off = _offsets(counts)
    pre = torch.full((P, 2 * I + _pad8(2 * I)), math.nan, dtype=dtype, device="cuda")[:, :2 * I]
    h = g.grouped_linear(x.cuda(), w.cuda(), off.cuda(), gated=True, pre=pre, out_dtype=torch.float32)
    want, size = ref.grouped(x, w, off)
    ref.assert_within(pre, want, ref.sum_bound(K) * size, "pre")
    ref.assert_within(h, *ref.gated(want, size, I, K), "h")
    plain = g.grouped_linear(x.cuda(), w.cuda(), off.cuda(), gated=True)
    assert torch.equal(plain, h.to(dtype))


def test_extreme_gates():
    # silu of large magnitudes: no NaN from exp's overflow
    x = torch.tensor([[400.0] * 8, [-400.0] * 8, [0.0] * 8], dtype=torch.float16)
    w = torch.ones(1, 16, 8, dtype=torch.float16)
    h = g.grouped_linear(x.cuda(), w.cuda(), torch.tensor([0, 3], dtype=torch.int32).cuda(), gated=True,
                         out_dtype=torch.float32)
    assert h[0, 0] == 3200.0 ** 2 and (h[1] == 0).all() and (h[2] == 0).all()


def test_no_terms_and_nothing_to_do():
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    x = torch.empty(5, 0, dtype=torch.float16, device="cuda")
    y = g.grouped_linear(x, torch.empty(2, 24, 0, dtype=torch.float16, device="cuda"), off)
    assert y.shape == (5, 24) and (y == 0).all()
    y = g.grouped_linear(torch.empty(0, 16, dtype=torch.float16, device="cuda"),
                         torch.zeros(2, 24, 16, dtype=torch.float16, device="cuda"), off * 0)
    assert y.shape == (0, 24)


def test_offsets_are_clamped():
    # offsets past the rows of x and y reach no memory outside them
    gen = torch.Generator().manual_seed(12)
    x = _randn(gen, 10, 32, dtype=torch.float16)
    w = _randn(gen, 2, 40, 32, dtype=torch.float16)
    off = torch.tensor([-4, 6, 500], dtype=torch.int32)
    want, size = ref.grouped(x, w, [0, 6, 10])
    y = g.grouped_linear(x.cuda(), w.cuda(), off.cuda())
    ref.assert_within(y, want, ref.sum_bound(32) * size)
    dw = g.grouped_weight_grad(x.cuda(), x.cuda(), off.cuda())
    for i, s in enumerate((slice(0, 6), slice(6, 10))):
        xs = x[s].double()
        ref.assert_within(dw[i], xs.T @ xs, ref.sum_bound(10) * (xs.abs().T @ xs.abs()))


@pytest.mark.parametrize("counts", COUNTS + [[63, 65, 1, 0, 127, 15, 16, 17]])
@pytest.mark.parametrize("N,K", [(200, 136), (129, 7), (1, 260), (64, 520)])
@pytest.mark.parametrize("out_dtype", [torch.float32, None])
def test_weight_grad(counts, N, K, out_dtype):
    dtype = torch.bfloat16 if N % 2 else torch.float16
    gen = torch.Generator().manual_seed(N + K)
    P = sum(counts) + 3
    dy, x = _randn(gen, P, N, dtype=dtype), _randn(gen, P, K, dtype=dtype)
    dy[-3:], x[-3:] = math.nan, math.inf       # positions of no group
    off = _offsets(counts)
    dw = g.grouped_weight_grad(_padded(dy, _pad8(N)), _padded(x, _pad8(K) + 8), off.cuda(),
                               out_dtype=out_dtype or dtype)
    assert g.gemm_get_device_status() == 0
    for e, c in enumerate(counts):
        s = slice(int(off[e]), int(off[e + 1]))
        a, b = dy[s].double(), x[s].double()
        ref.assert_within(dw[e], a.T @ b, ref.sum_bound(c) * (a.abs().T @ b.abs()), f"group {e}")


def test_weight_grad_keeps_other_groups_infinities_out():
    gen = torch.Generator().manual_seed(3)
    counts = [70, 1, 90, 5]
    off = _offsets(counts)
    dy, x = _randn(gen, 166, 72, dtype=torch.float16), _randn(gen, 166, 80, dtype=torch.float16)
    want = g.grouped_weight_grad(dy.cuda(), x.cuda(), off.cuda())
    dy[70], x[71:75] = math.inf, math.nan      # group 1's only row, the first of group 2
    got = g.grouped_weight_grad(dy.cuda(), x.cuda(), off.cuda())
    for e in (0, 3):
        assert torch.equal(got[e], want[e])


@pytest.mark.parametrize("H", [1, 7, 64, 1000])
@pytest.mark.parametrize("rows_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [1, 3, 8])
def test_combine_and_its_gradient(H, rows_dtype, k):
    gen = torch.Generator().manual_seed(H + k)
    T, E = 23, 6
    ids = torch.randint(-1, E, (T, k), generator=gen).int()
    ids[4] = -1                                 # a token without experts
    offsets, tokens, where = g.moe_plan(ids.cuda(), E)
    P = int(offsets[-1])
    rows = _randn(gen, T * k, H, dtype=rows_dtype)
    rows[P:] = math.nan                         # positions nobody has
    w = torch.randn(T, k, generator=gen)
    wh = where.cpu().long()
    live = (wh >= 0)[:, :, None]
    picked = torch.where(live, rows.double()[wh.clamp(min=0)], 0.0)
    y = g.moe_combine(rows.cuda(), where, w.cuda(), out_dtype=torch.float32)
    terms = picked * w.double()[:, :, None]
    ref.assert_within(y, terms.sum(1), (k + 1) * 2.0 ** -23 * terms.abs().sum(1), "combine")
    assert (y[4] == 0).all()
    s = g.moe_combine(rows.cuda(), where, out_dtype=torch.bfloat16)
    ref.assert_within(s, picked.sum(1), (k + 1) * 2.0 ** -23 * picked.abs().sum(1), "sum")

    dy = _randn(gen, T, H, dtype=torch.bfloat16)
    drows, dweights = g.moe_combine_backward(dy.cuda(), rows.cuda(), where, w.cuda())
    dots = picked * dy.double()[:, None, :]
    ref.assert_within(dweights, dots.sum(2), (H + 2) * 2.0 ** -23 * dots.abs().sum(2), "dweights")
    scaled = (w.double()[:, :, None] * dy.double()[:, None, :]).reshape(T * k, H)
    order = wh.reshape(-1)
    want = torch.zeros(P, H, dtype=torch.float64)
    want[order[order >= 0]] = scaled[order >= 0]
    ref.assert_within(drows[:P], want, 2.0 ** -24 * want.abs(), "drows")
    out = g.moe_dispatch(dy.cuda(), where)
    assert torch.equal(out[:P].cpu(), dy[tokens.cpu().long()[:P]])


@pytest.mark.parametrize("I", [1, 24, 129])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dh_dtype", [None, torch.float32])
def test_gated_silu_backward(I, dtype, dh_dtype):
    gen = torch.Generator().manual_seed(I)
    pre = (3 * _randn(gen, 37, 2 * I)).to(dtype)
    pre[0, 0], pre[1, 0] = 60000.0, -60000.0
    dh = _randn(gen, 37, I, dtype=dh_dtype or dtype)
    got = g.gated_silu_backward(pre.cuda(), dh.cuda())
    p = pre.double().requires_grad_(True)
    gate, up = p[:, :I], p[:, I:]
    (gate * torch.sigmoid(gate) * up).backward(dh.double())
    # a dozen fp32 roundings; 1 + gate (1 - s) cancels, its terms are at most 1 + |gate| (1 - s)
    s = torch.sigmoid(gate)
    size = torch.cat([dh.double().abs() * up.abs() * s * (1 + gate.abs() * (1 - s)),
                      dh.double().abs() * gate.abs() * s], 1).detach()
    ref.assert_within(got, p.grad, 16 * 2.0 ** -23 * size + 1e-30)
    # differences of the activation itself
    h = 1e-5
    d = torch.randn(37, 2 * I, generator=gen).double()
    act = lambda q: ((q[:, :I] * torch.sigmoid(q[:, :I]) * q[:, I:]) * dh.double())[2:].sum()  # noqa: E731
    diff = (act(pre.double() + h * d) - act(pre.double() - h * d)) / (2 * h)
    along = (got.double().cpu() * d)[2:].sum()
    room = (ref.ROUND[dtype] * 2 * size * d.abs())[2:].sum() + 1e-4 * (1 + diff.abs())
    assert abs(diff - along) <= room


def test_layer_gradient_against_differences():
    # the whole layer, routed: products, activation, weighted sum and all their gradients in a row
    gen = torch.Generator().manual_seed(21)
    T, E, k, H, I = 12, 5, 2, 16, 24
    dt = torch.float16
    x = _randn(gen, T, H, dtype=dt)
    w13 = (_randn(gen, E, 2 * I, H) * 0.3).to(dt)
    w2 = (_randn(gen, E, H, I) * 0.3).to(dt)
    logits = torch.randn(T, E, generator=gen)
    dy = _randn(gen, T, H, dtype=dt)
    ids, wt, off, tokens, where = g.moe_route(logits.cuda(), k)
    pre = torch.empty(T * k, 2 * I, dtype=dt, device="cuda")
    h = g.grouped_linear(x.cuda(), w13.cuda(), off, rows=tokens, gated=True, pre=pre)
    ys = g.grouped_linear(h, w2.cuda(), off, out_dtype=torch.float32)
    y = g.moe_combine(ys, where, wt, out_dtype=torch.float32)
    dys, dwt = g.moe_combine_backward(dy.cuda(), ys, where, wt)
    dh = g.grouped_linear(dys, w2.cuda(), off, opW="N", out_dtype=torch.float32)
    dw2 = g.grouped_weight_grad(dys, h, off)
    dpre = g.gated_silu_backward(pre, dh)
    dxs = g.grouped_linear(dpre, w13.cuda(), off, opW="N", out_dtype=torch.float32)
    dx = g.moe_combine(dxs, where, out_dtype=torch.float32)
    dw13 = g.grouped_weight_grad(dpre, g.moe_dispatch(x.cuda(), where), off)
    dlogits = g.moe_route_backward(dwt, logits.cuda(), ids)

    ids = ids.cpu().long()

    def loss(v):
        p = torch.gather(torch.softmax(v["logits"], 1), 1, ids)
        p = p / p.sum(1, keepdim=True)
        out = 0.0
        for j in range(k):
            a = torch.einsum("th,tih->ti", v["x"], v["w13"][ids[:, j]])
            act = torch.nn.functional.silu(a[:, :I]) * a[:, I:]
            out = out + p[:, j:j + 1] * torch.einsum("ti,thi->th", act, v["w2"][ids[:, j]])
        return out

    at = {"x": x.double(), "w13": w13.double(), "w2": w2.double(), "logits": logits.double()}
    # 16-bit roundings of h, dys and dpre: three relative errors of 2^-11 in sums of random signs
    want_y = loss(at)
    assert (y.double().cpu() - want_y).norm() <= 4 * 2.0 ** -11 * want_y.norm()
    got = {"x": dx, "w13": dw13, "w2": dw2, "logits": dlogits}
    for name, grad in got.items():
        d = grad.double().cpu()
        d = d / d.norm()                         # steepest direction: the difference is its norm
        step = 1e-5
        hi = (loss({**at, name: at[name] + step * d}) * dy.double()).sum()
        lo = (loss({**at, name: at[name] - step * d}) * dy.double()).sum()
        diff = (hi - lo) / (2 * step)
        assert abs(diff - grad.double().norm().cpu()) <= 4 * 2.0 ** -11 * diff.abs(), name


def test_graph_capture_and_streams():
    gen = torch.Generator().manual_seed(30)
    T, E, k, H, I = 40, 8, 2, 64, 48
    x = _randn(gen, T, H, dtype=torch.bfloat16).cuda()
    w13 = _randn(gen, E, 2 * I, H, dtype=torch.bfloat16).cuda()
    w2 = _randn(gen, E, H, I, dtype=torch.bfloat16).cuda()
    logits = torch.randn(T, E, generator=gen).cuda()

    def layer():
        ids, wt, off, tokens, where = g.moe_route(logits, k)
        h = g.grouped_linear(x, w13, off, rows=tokens, gated=True)
        return g.moe_combine(g.grouped_linear(h, w2, off, out_dtype=torch.float32), where, wt)

    want = layer()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            other = layer()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    logits.copy_(logits.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, layer())
