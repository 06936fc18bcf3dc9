"""What the training operators of this library's linear layers are measured on.

Block-scaled 8-bit values (written and read back), products of them (a linear layer's forward pass, its
input's and its weight's gradient), and the orthogonalised update of a weight.  ``run`` computes a case in
elementary torch operations in fp32 (``own`` false) or through the library's entry points (``own`` true);
``exact`` computes it in fp64.

A block of 128 values along an axis, or of 128 x 128, shares one fp32 scale: the smallest power of two s,
at least 2^-126, with max|x| <= s * m, m the largest 8-bit value (448 for e4m3, 57344 for e5m2), and 1 for a
block of zeros; a value is stored as x / s rounded to the nearest 8-bit value, ties to even.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_EIGHT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_BLOCKS = {"rows": (1, 128), "columns": (128, 1), "tiles": (128, 128)}


# --------------------------------------------------------------------------- the cases
def _quant(name, rows, cols, block, dtype, eight="e4m3"):
    return dict(name=name, kind="quant", rows=rows, cols=cols, block=block, dtype=dtype, eight=eight)


def _linear(name, tokens, n, k, dtype, kind="linear", eight="e4m3"):
    return dict(name=name, kind=kind, tokens=tokens, n=n, k=k, dtype=dtype, eight=eight)


def _update(name, count, n, k, dtype, rank):
    return dict(name=name, kind="update", count=count, n=n, k=k, dtype=dtype, rank=rank)


def listed():
    return [
        # the activations of a decoding batch, quantised along their rows and read back: latency
        _quant("quant_decode", 64, 4096, "rows", "bf16"),
        # a training batch's activations, kept for the forward product and for the weight's gradient
        _quant("quant_both", 8191, 4096, "both", "bf16"),
        # one request decoding alone: the 8-bit weight is read once
        _linear("linear_token", 1, 4096, 4096, "bf16"),
        # a decoding batch on a wide layer
        _linear("linear_decode", 64, 8192, 4096, "bf16"),
        # a ragged batch on a layer of odd sizes
        _linear("linear_ragged", 1001, 2309, 2500, "f16"),
        # a prompt batch on the linear layer of this repository's workloads
        _linear("linear_prompt", 16384, 4096, 4096, "bf16"),
        # the layer's backward pass (gradients of input and weight): a small odd batch, wide-range type
        _linear("grad_small", 333, 1040, 520, "bf16", "linear_grad", "e5m2"),
        # the same for a training batch
        _linear("grad_batch", 8192, 4096, 4096, "bf16", "linear_grad"),
        # the optimiser's update of one small projection
        _update("update_small", 1, 256, 512, "f32", 32),
        # of a stack of the experts' tall matrices
        _update("update_experts", 16, 1000, 520, "bf16", 128),
        # of one wide matrix
        _update("update_wide", 1, 2048, 4096, "bf16", 512),
        # of a large square one
        _update("update_square", 1, 4096, 4096, "f32", 1024),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm; the large ones odd."""
    n = min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n if n < 1000 else (n - 1) | 1


def draw(rng):
    kind = rng.choice(["quant", "linear", "linear", "linear_grad", "update", "update"])
    if kind == "quant":
        c = _quant("", _log(rng, 1, 16384), _log(rng, 16, 8192), rng.choice(["rows", "tiles", "columns", "both"]),
                   rng.choice(["bf16", "bf16", "f16", "f32"]), rng.choice(["e4m3", "e4m3", "e5m2"]))
    elif kind == "linear":
        c = _linear("", _log(rng, 1, 16384), _log(rng, 64, 8192), _log(rng, 128, 8192), rng.choice(["bf16", "bf16", "f16"]))
    elif kind == "linear_grad":
        c = _linear("", _log(rng, 16, 8192), _log(rng, 128, 4096), _log(rng, 128, 4096), "bf16", kind,
                    rng.choice(["e4m3", "e5m2"]))
    else:
        n, k = _log(rng, 16, 4096), _log(rng, 16, 4096)
        small = min(n, k)
        most = max(1, min(16, 4096 ** 3 // (n * k * small), (1 << 25) // (n * k)))
        c = _update("", _log(rng, 1, most), n, k, rng.choice(["bf16", "f32", "f16"]), max(1, small // rng.choice([1, 2, 4, 8])))
    if kind in ("linear", "linear_grad"):  # no more work than the largest listed case
        most = 16384 * 4096 * 4096 if kind == "linear" else 8192 * 4096 * 4096
        c["tokens"] = max(1, min(c["tokens"], most // (c["n"] * c["k"])))
    del c["name"]
    return c


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _activations(g, rows, cols, dtype, std=1.0):
    """Normal values whose columns differ in size, as a layer's channels do."""
    size = torch.exp(0.7 * torch.randn(cols, generator=g, device="cuda"))
    return _randn(g, rows, cols).mul_(size).mul_(std).to(dtype)


def _stored(q):
    """The matrix with rows on 16-byte boundaries, as a checkpoint's loader lays it out."""
    out = torch.zeros(q.shape[0], (q.shape[1] + 15) // 16 * 16, dtype=torch.uint8, device=q.device).view(q.dtype)
    out.view(torch.uint8)[:, :q.shape[1]] = q.view(torch.uint8)
    return out[:, :q.shape[1]]


def prepare(case, seed):
    c, g = case, _gen(seed)
    dt = _TYPES[c["dtype"]]
    s = {"case": c}
    if c["kind"] == "quant":
        s["x"] = _activations(g, c["rows"], c["cols"], dt)
    elif c["kind"] in ("linear", "linear_grad"):
        w = _randn(g, c["n"], c["k"], std=c["k"] ** -0.5)
        q, s["w_scales"] = _plain_quantize(w, (128, 128), "e4m3")
        s["w"] = _stored(q)
        if c["kind"] == "linear":
            s["x"] = _activations(g, c["tokens"], c["k"], dt)
        else:  # the gradient of the layer's output, and what the forward pass kept of its input
            s["dy"] = _activations(g, c["tokens"], c["n"], dt, std=1e-3)
            q, s["x_scales"] = _plain_quantize(_activations(g, c["tokens"], c["k"], dt), (128, 1), "e4m3")
            s["x"] = _stored(q)
    else:  # a gradient: a strong part of low rank and noise below it
        a = _randn(g, c["count"], c["n"], c["rank"])
        b = _randn(g, c["count"], c["rank"], c["k"], std=c["rank"] ** -0.5)
        a *= torch.exp(-3.0 * torch.arange(c["rank"], device="cuda") / c["rank"])
        noise = _randn(g, c["count"], c["n"], c["k"], std=0.05)
        s["g"] = torch.baddbmm(noise, a, b).mul_(1e-3).to(dt)
        if c["count"] == 1:
            s["g"] = s["g"][0]
    return s


# --------------------------------------------------------------------------- the plain forms
def _plain_scales(amax):
    m, e = torch.frexp(amax)  # both types' largest value is 1.75 times a power of two
    return e + (m > 0.875).int()


def _plain_quantize(x, block, eight):
    """(8-bit matrix, scales) of x."""
    r, c = x.shape
    b0, b1 = block
    nr, nc = -(-r // b0), -(-c // b1)
    v = x.new_zeros(nr * b0, nc * b1, dtype=torch.float32)
    v[:r, :c] = x
    v = v.reshape(nr, b0, nc, b1)
    amax = v.abs().amax(dim=(1, 3))
    power = _plain_scales(amax) - (9 if eight == "e4m3" else 16)
    power = torch.clamp(power, min=-126) * (amax > 0)
    scales = ((power + 127) << 23).view(torch.float32)  # 2 ** power
    q = (v / scales[:, None, :, None]).to(_EIGHT[eight])
    return q.reshape(nr * b0, nc * b1)[:r, :c], scales


def _plain_values(q, scales):
    """The fp32 values that an 8-bit matrix and its scales stand for."""
    r, c = q.shape
    b0, b1 = (1 if scales.shape[0] == r else 128), (1 if scales.shape[1] == c else 128)
    i = torch.div(torch.arange(r, device=q.device), b0, rounding_mode="floor")
    j = torch.div(torch.arange(c, device=q.device), b1, rounding_mode="floor")
    return q.float() * scales[i][:, j]


def _plain_quant(s):
    c, out = s["case"], {}
    for way in ("rows", "columns") if c["block"] == "both" else (c["block"],):
        q, scales = _plain_quantize(s["x"], _BLOCKS[way], c["eight"])
        out[way] = _plain_values(q, scales).to(s["x"].dtype)
        out[way + "_scales"] = scales
    return out


def _plain_linear(s):
    x = _plain_values(*_plain_quantize(s["x"], (1, 128), s["case"]["eight"]))
    return {"y": (x @ _plain_values(s["w"], s["w_scales"]).T).to(s["x"].dtype)}


def _plain_linear_grad(s):
    eight, dt = s["case"]["eight"], s["dy"].dtype
    rows = _plain_values(*_plain_quantize(s["dy"], (1, 128), eight))
    columns = _plain_values(*_plain_quantize(s["dy"], (128, 1), eight))
    dx = rows @ _plain_values(s["w"], s["w_scales"])
    return {"dx": dx.to(dt), "dw": columns.T @ _plain_values(s["x"], s["x_scales"])}


def _plain_step(x, a, b, c):
    gram = x @ x.transpose(1, 2)
    return a * x + (b * gram + c * (gram @ gram)) @ x


def _plain_update(s):
    x = s["g"].float().reshape(s["case"]["count"], s["case"]["n"], s["case"]["k"])
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + 1e-7)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = _plain_step(_plain_step(x, *_COEFFICIENTS), *_COEFFICIENTS)
    x = _plain_step(_plain_step(_plain_step(x, *_COEFFICIENTS), *_COEFFICIENTS), *_COEFFICIENTS)
    if tall:
        x = x.transpose(1, 2)
    return {"update": x.reshape(s["g"].shape).to(torch.bfloat16)}


_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


# --------------------------------------------------------------------------- the library's operators
def _own(s):
    import dense_gemm_sgemm_gb300 as g

    c = s["case"]
    if c["kind"] == "update":
        return {"update": g.orthogonalize(s["g"])}
    eight = _EIGHT[c["eight"]]
    if c["kind"] == "quant":
        dt = s["x"].dtype
        if c["block"] == "both":
            q, scales, qc, scalesc = g.quantize_both(s["x"], dtype=eight)
            return {"rows": g.dequantize_blocks(q, scales, out_dtype=dt), "rows_scales": scales,
                    "columns": g.dequantize_blocks(qc, scalesc, out_dtype=dt), "columns_scales": scalesc}
        q, scales = g.quantize_blocks(s["x"], _BLOCKS[c["block"]], dtype=eight)
        return {c["block"]: g.dequantize_blocks(q, scales, out_dtype=dt), c["block"] + "_scales": scales}
    if c["kind"] == "linear":
        x, scales = g.quantize_blocks(s["x"], dtype=eight)
        return {"y": g.scaled_matmul(x, scales, s["w"], s["w_scales"], out_dtype=s["x"].dtype)}
    q, scales, qc, scalesc = g.quantize_both(s["dy"], dtype=eight)
    dx = g.scaled_matmul(q, scales, s["w"], s["w_scales"], opB="N", out_dtype=s["dy"].dtype)
    dw = g.scaled_matmul(qc, scalesc, s["x"], s["x_scales"], opA="T", opB="N", out_dtype=torch.float32)
    return {"dx": dx, "dw": dw}


def run(state):
    if own:
        return _own(state)
    return {"quant": _plain_quant, "linear": _plain_linear, "linear_grad": _plain_linear_grad,
            "update": _plain_update}[state["case"]["kind"]](state)


# --------------------------------------------------------------------------- floors
def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    if c["kind"] == "quant":
        ways = 2 if c["block"] == "both" else 1
        n = c["rows"] * c["cols"]
        return {"bytes": n * (size + ways * (2 + size)), "flops": 4 * ways * n}
    if c["kind"] == "update":
        n, k = min(c["n"], c["k"]), max(c["n"], c["k"])  # the Gram matrix and its square are symmetric
        return {"bytes": c["count"] * n * k * (size + 2), "flops": c["count"] * 5 * (3 * n * n * k + n * n * n)}
    t, n, k = c["tokens"], c["n"], c["k"]
    if c["kind"] == "linear":
        return {"bytes": 2 * t * k + n * k + 2 * t * n, "flops": 2 * t * n * k}
    return {"bytes": 2 * t * n + n * k + t * k + 2 * t * k + 4 * n * k, "flops": 4 * t * n * k}


# --------------------------------------------------------------------------- in 64 bits
def _two_to(power):
    return ((power.long() + 1023) << 52).view(torch.float64)


def _exact_values(x, block, eight):
    """(values, scales) of x in blocks: scales by powers of two tried from the smallest, values on their grid."""
    x = x.double()
    r, c = x.shape
    most, mantissa, least = (448.0, 3, -6) if eight == "e4m3" else (57344.0, 2, -14)
    rows = torch.arange(r, device=x.device) // block[0]
    cols = torch.arange(c, device=x.device) // block[1]
    index = rows[:, None] * (int(cols[-1]) + 1) + cols[None, :]
    count = (int(rows[-1]) + 1) * (int(cols[-1]) + 1)
    amax = x.new_zeros(count).scatter_reduce_(0, index.reshape(-1), x.abs().reshape(-1), "amax")
    power = torch.floor(torch.log2(amax.clamp(min=2.0 ** -200))) - 20.0
    power = torch.clamp(power, min=-126.0)
    for _ in range(24):
        power = torch.where(amax > _two_to(power) * most, power + 1.0, power)
    scale = torch.where(amax > 0, _two_to(power), 1.0)
    full = scale[index]
    y = x / full
    exponent = torch.frexp(y).exponent - 1
    step = _two_to(torch.clamp(exponent, min=least) - mantissa)
    return torch.round(y / step) * step * full, scale.reshape(int(rows[-1]) + 1, int(cols[-1]) + 1)


def _exact_stored(q, scales):
    """The values of a stored 8-bit matrix."""
    r, c = q.shape
    full = scales.double()
    if scales.shape[0] != r:
        full = full.repeat_interleave(128, dim=0)[:r]
    if scales.shape[1] != c:
        full = full.repeat_interleave(128, dim=1)[:, :c]
    return q.to(torch.float64) * full


def exact(case, seed):
    s = prepare(case, seed)
    c, kind = case, case["kind"]
    if kind == "quant":
        out = {}
        for way in ("rows", "columns") if c["block"] == "both" else (c["block"],):
            out[way], out[way + "_scales"] = _exact_values(s["x"], _BLOCKS[way], c["eight"])
        return out
    if kind == "linear":
        x = _exact_values(s["x"], (1, 128), c["eight"])[0]
        return {"y": torch.einsum("tk,nk->tn", x, _exact_stored(s["w"], s["w_scales"]))}
    if kind == "linear_grad":
        w, x = _exact_stored(s["w"], s["w_scales"]), _exact_stored(s["x"], s["x_scales"])
        return {"dx": torch.einsum("tn,nk->tk", _exact_values(s["dy"], (1, 128), c["eight"])[0], w),
                "dw": torch.einsum("tn,tk->nk", _exact_values(s["dy"], (128, 1), c["eight"])[0], x)}
    out = []
    for g in s["g"].double().reshape(c["count"], c["n"], c["k"]):
        x = g / (torch.linalg.norm(g) + 1e-7)
        # odd polynomial of the singular values, five times over, from the smaller side
        flip = c["n"] > c["k"]
        x = x.mT.contiguous() if flip else x
        for _ in range(5):
            gram = torch.mm(x, x.mT)
            eye = torch.eye(gram.shape[0], dtype=torch.float64, device=x.device)
            inner = _COEFFICIENTS[1] * eye + _COEFFICIENTS[2] * gram
            x = torch.mm(_COEFFICIENTS[0] * eye + torch.mm(inner, gram), x)
        out.append(x.mT if flip else x)
    return {"update": torch.stack(out).reshape(s["g"].shape)}
