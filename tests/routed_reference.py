"""Plain 64-bit forms of the routed products, and error bounds for their tests.

Bounds.  A product of 16-bit inputs is exact in fp32's range and its sum is kept in fp32: the tensor
cores add blocks of at least 8 products, each addition losing at most 2^-22 of the running sum of
magnitudes (a truncated addition, two bits of headroom), and at most 32 more additions join the
blocks' lanes, parts of K and adapter ranks; so |sum - exact| <= (K / 8 + 32) 2^-22 sum|x w|.
Rounding to the output type adds its unit roundoff times the magnitude, 2^-8 for bf16, 2^-11 for
fp16, 2^-24 for fp32, and half the spacing of the smallest numbers, 2^-25 for fp16.
"""
import numpy as np
import torch

ROUND = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-38, torch.float16: 2.0 ** -25, torch.bfloat16: 1e-38}


def sum_bound(K):
    return (K / 8 + 32) * 2.0 ** -22


def assert_within(got, ref, bound, what=""):
    """|got - ref| <= bound + the rounding of got's type, everywhere; got has no NaN."""
    g = got.detach().double().cpu()
    bound = bound + ROUND[got.dtype] * (ref.abs() + bound) + TINY[got.dtype]
    err = (g - ref).abs()
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bound, first at {i}: "
                             f"got {g[i].item()} wanted {ref[i].item()} +- {bound[i].item()}")


def order(values, count):
    """Indices of the `count` largest values that are not -inf, ties to the lowest index."""
    idx = sorted((i for i in range(len(values)) if values[i] > -np.inf), key=lambda i: (-values[i], i))
    return idx[:count]


def scores(x, score):
    live = x > -np.inf
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(live, 1.0 / (1.0 + np.exp(-np.where(live, x, 0.0))), 0.0)
    if not live.any():
        return np.zeros_like(x)
    e = np.where(live, np.exp(np.where(live, x, 0.0) - x[live].max()), 0.0)
    return e / e.sum()


def route(logits, top_k, bias=None, score="softmax", groups=1, groups_kept=1, group_top=1,
          renormalise=True, scale=1.0):
    """(ids, weights) by the definition, one row at a time."""
    x = logits.double().cpu().numpy().copy()
    x[np.isnan(x)] = -np.inf
    x = np.minimum(x, np.finfo(np.float32).max)
    T, E = x.shape
    b = None if bias is None else bias.double().cpu().numpy()
    ids = -np.ones((T, top_k), dtype=np.int64)
    weights = np.zeros((T, top_k))
    for t in range(T):
        s = scores(x[t], score)
        live = x[t] > -np.inf
        value = np.where(live, s if b is None else s + b, -np.inf)
        value[np.isnan(value)] = -np.inf
        choice = x[t].copy() if b is None else value.copy()
        if groups > 1:
            run = value.reshape(groups, -1)
            best = np.full(groups, -np.inf)
            for g in range(groups):
                top = sorted(run[g][run[g] > -np.inf], reverse=True)[:group_top]
                if top:
                    best[g] = sum(top)
            keep = order(best, groups_kept)
            for g in range(groups):
                if g not in keep:
                    choice.reshape(groups, -1)[g] = -np.inf
        pick = order(choice, top_k)
        w = s[pick]
        if renormalise:
            w = w / w.sum() if w.sum() > 0 else 0.0 * w
        ids[t, :len(pick)] = pick
        weights[t, :len(pick)] = w * scale
    return torch.from_numpy(ids), torch.from_numpy(weights)


def plan(ids, experts):
    """offsets, tokens, where by the definition (tokens only up to offsets[experts])."""
    T, k = ids.shape
    flat = [int(e) for e in ids.reshape(-1)]
    where = [-1] * (T * k)
    tokens, offsets = [], [0]
    for e in range(experts):
        for s in range(T * k):
            if flat[s] == e:
                where[s] = len(tokens)
                tokens.append(s // k)
        offsets.append(len(tokens))
    return torch.tensor(offsets), torch.tensor(tokens, dtype=torch.int64), torch.tensor(where).reshape(T, k)


def grouped(x, w, offsets, rows=None, opW="T"):
    """(product, sum of magnitudes) in 64 bits, zeros at positions of no group."""
    off = [int(v) for v in offsets]
    n = x.shape[0] if rows is None else rows.numel()
    x = x.double().cpu()
    if rows is not None:
        r = rows.long().cpu()
        ok = (r >= 0) & (r < x.shape[0])
        x = torch.where(ok[:, None], x[r.clamp(0, max(x.shape[0] - 1, 0))], 0.0)
    w = w.double().cpu()
    if opW == "T":
        w = w.transpose(1, 2)
    y = torch.zeros(n, w.shape[2], dtype=torch.float64)
    m = torch.zeros_like(y)
    for g in range(w.shape[0]):
        s = slice(off[g], off[g + 1])
        y[s] = x[s] @ w[g]
        m[s] = x[s].abs() @ w[g].abs()
    return y, m


def gated(pre, magnitude, I, K):
    """(h, bound of its fp32 evaluation) of [gate | up] and the magnitudes of their sums."""
    g, u = pre[:, :I], pre[:, I:]
    eg, eu = sum_bound(K) * magnitude[:, :I], sum_bound(K) * magnitude[:, I:]
    silu = g * torch.sigmoid(g)
    # |silu'| <= 1.1; the exponential, division and products lose a few 2^-24 each
    return silu * u, 1.1 * u.abs() * eg + (silu.abs() + 1.1 * eg) * eu + 16 * 2.0 ** -24 * (silu * u).abs()
