"""The block-scaled products and the update record no gradient and say so."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import dense_gemm_sgemm_gb300 as g

    g.load()
    return g


def test_tensors_that_require_a_gradient_are_refused(g):
    x = torch.randn(40, 256, device="cuda")
    q, s = g.quantize_blocks(x)
    leaf, scales = x.clone().requires_grad_(), s.clone().requires_grad_()
    calls = [lambda: g.quantize_blocks(leaf), lambda: g.quantize_both(leaf), lambda: g.orthogonalize(leaf), lambda: g.orthogonalize(leaf * 2),
             lambda: g.dequantize_blocks(q, scales), lambda: g.scaled_matmul(q, scales, q, s), lambda: g.scaled_matmul(q, s, q, scales)]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call()
    with torch.no_grad():  # as in a layer's own forward and backward, or an optimiser
        for call in calls:
            call()
    assert torch.equal(g.orthogonalize(leaf.detach()), g.orthogonalize(x))


def test_inside_an_autograd_function(g):
    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            q, s, ctx.columns, ctx.column_scales = g.quantize_both(x)
            ctx.w, ctx.w_scales = g.quantize_blocks(w, (128, 128))
            return g.scaled_matmul(q, s, ctx.w, ctx.w_scales, out_dtype=torch.float32)

        @staticmethod
        def backward(ctx, dy):
            q, s, columns, scales = g.quantize_both(dy)
            return (g.scaled_matmul(q, s, ctx.w, ctx.w_scales, opB="N", out_dtype=torch.float32),
                    g.scaled_matmul(columns, scales, ctx.columns, ctx.column_scales, opA="T", opB="N", out_dtype=torch.float32))

    r = torch.Generator().manual_seed(2)
    # whole numbers up to 8, which 8 bits hold, and sums that fp32 holds: exact
    x, w, dy = (torch.randint(-8, 9, shape, generator=r).float().cuda() for shape in ((100, 300), (50, 300), (100, 50)))
    x.requires_grad_(), w.requires_grad_()
    y = Linear.apply(x, w)
    y.backward(dy)
    assert torch.equal(y, x.detach() @ w.detach().T) and torch.equal(x.grad, dy @ w.detach()) and torch.equal(w.grad, dy.T @ x.detach())
