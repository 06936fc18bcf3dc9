"""Plain forms of the block-scaled 8-bit operators in 64 bits, and the bounds their results are held to.

quantise()   scales and codes by the definition; codes and scales are unique, so they are compared bit for bit.
product()    (C, bound): the value in fp64 and how far a result may be off.  A block's products are exact and
             summed in fp32 in some order, with an error of at most one step (2^-23) an addition; blocks are
             added in fp32: over all (128 + blocks + 4) steps of the sum of magnitudes.  The result is rounded
             once, by half a step of its type.
"""
import torch

MOST = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def expand(scales, shape, block):
    return scales.double().repeat_interleave(block[0], 0)[:shape[0]].repeat_interleave(block[1], 1)[:, :shape[1]]


def block_of(scales, shape):
    return tuple(128 if n == -(-size // 128) else 1 for n, size in zip(scales.shape, shape))


def quantise(x, block, dtype):
    """(codes as uint8, scales) on the CPU."""
    x = x.detach().cpu().double()
    rows, cols = x.shape
    down, across = -(-rows // block[0]), -(-cols // block[1])
    padded = torch.zeros(down * block[0], across * block[1], dtype=torch.float64)
    padded[:rows, :cols] = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    amax = padded.reshape(down, block[0], across, block[1]).amax((1, 3))
    _, e = torch.frexp(amax / MOST[dtype])
    # amax / most = m 2^e, m in [1/2, 1): the smallest power of two at least that large
    power = torch.where(amax == MOST[dtype] * 2.0 ** (e - 1).double(), e - 1, e).clamp(min=-126)
    scales = torch.where(amax > 0, 2.0 ** power.double(), torch.ones_like(amax))
    v = x / expand(scales, x.shape, block)
    v = torch.where(torch.isfinite(x), v, torch.full_like(v, float("nan")))
    # exact in fp32 down to its subnormals, far below both types' smallest value
    codes = v.float().to(dtype).view(torch.uint8)
    codes = torch.where(torch.isnan(v), torch.full_like(codes, 0x7F), codes)
    return codes, scales.float()


def values(q, scales):
    return q.to(torch.float32).double() * expand(scales, q.shape, block_of(scales, q.shape))


def product(A, sa, B, sb, opA="N", opB="T", dtype=torch.float32):
    a, b = values(A, sa), values(B, sb)
    a = a if opA == "N" else a.T
    b = b if opB == "N" else b.T
    c, size = a @ b, a.abs() @ b.abs()
    steps = 128 + -(-a.shape[1] // 128) + 4
    return c, steps * 2.0 ** -23 * size + HALF_STEP[dtype] * c.abs() + TINY[dtype]


def stored(q):
    """A copy with rows on 16-byte boundaries."""
    out = torch.zeros(q.shape[0], -(-q.shape[1] // 16) * 16 or 16, dtype=torch.uint8, device=q.device)
    out[:, :q.shape[1]] = q.view(torch.uint8)
    return out.view(q.dtype)[:, :q.shape[1]]


def operand(g, mn, K, op_k_first, mn_block, dtype, ints=True, spread=2):
    """A random stored matrix of mn x K (or K x mn) and its scales: small whole numbers (exact sums), or any codes."""
    shape = (K, mn) if op_k_first else (mn, K)
    if ints:
        q = torch.randint(-4, 5, shape, generator=g).float()
    else:
        q = torch.randn(shape, generator=g) * 20
    q = stored(q.to(dtype))
    blocks = (-(-K // 128), -(-mn // mn_block))
    scales = 2.0 ** torch.randint(-spread, spread + 1, blocks, generator=g).float()
    if not ints:
        scales *= 0.5 + torch.rand(blocks, generator=g)
    return q, scales if op_k_first else scales.T
