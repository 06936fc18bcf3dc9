"""What the routed operators of this library are measured on.

Products whose weights differ from row to row: a router that gives each token its experts, the
experts' products with the gated activation between them and the weighted sum behind them, and a
shared projection with a low-rank adapter of each request beside it.  ``run`` computes a case in
elementary torch operations in fp32 (``own`` false) or through the library's entry points (``own``
true); ``exact`` computes it in fp64.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# --------------------------------------------------------------------------- the cases
def _route(name, tokens, experts, top_k, score, dtype, bias=False, groups=1, kept=1, group_top=1,
           renormalise=True, scale=1.0, kind="route"):
    return dict(name=name, kind=kind, tokens=tokens, experts=experts, top_k=top_k, score=score,
                dtype=dtype, bias=bias, groups=groups, kept=kept, group_top=group_top,
                renormalise=renormalise, scale=scale)


def _experts(name, tokens, experts, top_k, hidden, inner, dtype, skew=0.0, kind="experts"):
    return dict(name=name, kind=kind, tokens=tokens, experts=experts, top_k=top_k, hidden=hidden,
                inner=inner, dtype=dtype, skew=skew)


def _lora(name, tokens, requests, adapters, rank, n, k, dtype):
    return dict(name=name, kind="lora", tokens=tokens, requests=requests, adapters=adapters,
                rank=rank, n=n, k=k, dtype=dtype)


def listed():
    return [
        # the router of one decoding step of eight requests: latency is all of it
        _route("route_step", 8, 64, 8, "softmax", "f32"),
        # the router of a long prompt batch: sigmoid scores, a balancing bias, half of the groups
        _route("route_prompt", 16384, 256, 8, "sigmoid", "f32", bias=True, groups=8, kept=4,
               group_top=2, scale=2.5),
        # the same router's backward pass in training, weights not renormalised, an odd batch
        _route("route_grad", 8191, 128, 6, "softmax", "bf16", renormalise=False, kind="route_grad"),
        # one request decoding alone: the chosen experts' weights are read once each
        _experts("experts_token", 1, 64, 8, 2048, 1024, "bf16"),
        # a decoding batch: nearly every expert is read for a few rows
        _experts("experts_decode", 64, 128, 8, 2048, 1024, "bf16", skew=0.5),
        # a batch of ragged sizes, experts of uneven load, narrow rows
        _experts("experts_ragged", 777, 24, 3, 1000, 520, "f16", skew=1.0),
        # a prompt batch: the products are bound by the tensor cores
        _experts("experts_prompt", 8192, 64, 4, 2048, 1024, "bf16", skew=0.5),
        # training, backward through the weighted sum and the second product: a small odd batch
        _experts("experts_grad_small", 333, 16, 2, 1024, 512, "f16", skew=1.0, kind="experts_grad"),
        # the same for a training batch
        _experts("experts_grad", 8192, 32, 4, 2048, 1024, "bf16", skew=0.5, kind="experts_grad"),
        # 64 requests decoding one token each, every one with an adapter of its own
        _lora("lora_decode", 64, 64, 64, 16, 4096, 4096, "bf16"),
        # prompts and single tokens of 40 requests in one batch, some without an adapter
        _lora("lora_mixed", 1001, 40, 24, 32, 2560, 2304, "bf16"),
        # a few long prompts on the linear layer of this repository's workloads
        _lora("lora_prompt", 8192, 7, 8, 64, 4096, 4096, "f16"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm; the large ones odd."""
    n = min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n if n < 1000 else (n - 1) | 1


def draw(rng):
    kind = rng.choice(["route", "route_grad", "experts", "experts", "experts_grad", "lora", "lora"])
    if kind in ("route", "route_grad"):
        experts = 8 * rng.randint(1, 32)
        top_k = rng.randint(1, 8)
        score = rng.choice(["softmax", "sigmoid"])
        groups = rng.choice([1, 1, 2, 4, 8]) if kind == "route" and experts >= 64 else 1
        kept = rng.randint((groups + 1) // 2, groups)
        return _route_case(kind, _log(rng, 1, 16384), experts, top_k, score,
                           rng.choice(["f32", "f32", "bf16", "f16"]),
                           score == "sigmoid" and kind == "route" and rng.random() < 0.7, groups, kept,
                           rng.choice([1, 2]) if groups > 1 else 1, rng.random() < 0.6,
                           rng.choice([1.0, 2.5]))
    if kind in ("experts", "experts_grad"):
        hidden, inner = 8 * rng.randint(32, 256), 8 * rng.randint(16, 128)
        experts = rng.randint(4, 64 if kind == "experts" else 32)
        top_k = rng.randint(1, 4)
        tokens = _log(rng, 1 if kind == "experts" else 16, 8192)
        c = _experts("", tokens, experts, top_k, hidden, inner, rng.choice(["bf16", "f16"]),
                     rng.choice([0.0, 0.5, 1.0]), kind)
    else:
        tokens = _log(rng, 1, 8192)
        requests = min(tokens, _log(rng, 1, 128))
        c = _lora("", tokens, requests, rng.randint(1, 64), 8 * rng.randint(1, 8),
                  8 + 16 * rng.randint(16, 255), 8 + 16 * rng.randint(16, 255),
                  rng.choice(["bf16", "f16"]))
    del c["name"]
    return c


def _route_case(kind, *a):
    tokens, experts, top_k, score, dtype, bias, groups, kept, group_top, renormalise, scale = a
    if experts % groups:
        groups, kept, group_top = 1, 1, 1
    c = _route("", tokens, experts, min(top_k, experts // groups * kept), score, dtype, bias, groups,
               kept, group_top, renormalise, scale, kind)
    del c["name"]
    return c


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
    return x.mul_(std).to(dtype)


def _weights(g, *shape, dtype, std):
    """Large weights, made in their own type."""
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def _ids(c, g):
    """Distinct experts of each token, drawn without replacement from uneven popularities."""
    pop = torch.randn(c["experts"], generator=g, device="cuda") * c["skew"]
    u = torch.rand(c["tokens"], c["experts"], generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    return torch.topk(pop - torch.log(-torch.log(u)), min(c["top_k"], c["experts"]), dim=1).indices


def _plan_of(ids, experts):
    """offsets [experts + 1], tokens [T k] (position -> token), where [T, k] (slot -> position)."""
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    where = torch.empty_like(order)
    where[order] = torch.arange(order.numel(), device=order.device)
    bounds = torch.arange(experts + 1, device=order.device)
    offsets = torch.searchsorted(flat[order], bounds)
    tokens = torch.div(order, ids.shape[1], rounding_mode="floor")
    return offsets.int(), tokens.int(), where.reshape(ids.shape).int()


def prepare(case, seed):
    c, g = case, _gen(seed)
    dt = _TYPES[c["dtype"]]
    s = {"case": c}
    if c["kind"] in ("route", "route_grad"):
        s["logits"] = _randn(g, c["tokens"], c["experts"], dtype=dt, std=1.5)
        # a balancing bias moves in steps of a thousandth
        s["bias"] = torch.round(_randn(g, c["experts"], std=50.0)) * 1e-3 if c["bias"] else None
        if c["kind"] == "route_grad":
            s["ids"] = torch.topk(s["logits"].float(), c["top_k"], dim=1).indices.int()
            s["dweights"] = _randn(g, c["tokens"], c["top_k"])
    elif c["kind"] in ("experts", "experts_grad"):
        ids = _ids(c, g)
        s["offsets"], s["tokens"], s["where"] = _plan_of(ids, c["experts"])
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        s["weights"] = torch.softmax(_randn(g, *ids.shape), dim=1)
        h, i = c["hidden"], c["inner"]
        s["w2"] = _weights(g, c["experts"], h, i, dtype=dt, std=i ** -0.5)
        if c["kind"] == "experts":
            s["x"] = _randn(g, c["tokens"], h, dtype=dt)
            s["w13"] = _weights(g, c["experts"], 2 * i, h, dtype=dt, std=h ** -0.5)
        else:  # what the forward pass kept: the second product's input and output
            s["dy"] = _randn(g, c["tokens"], h, dtype=dt)
            s["inner"] = _randn(g, ids.numel(), i, dtype=dt)
            s["ys"] = _randn(g, ids.numel(), h)
    else:
        n, k, r = c["n"], c["k"], c["rank"]
        s["x"] = _randn(g, c["tokens"], k, dtype=dt)
        s["w"] = _weights(g, n, k, dtype=dt, std=k ** -0.5)
        s["a"] = _weights(g, c["adapters"], r, k, dtype=dt, std=k ** -0.5)
        s["b"] = _weights(g, c["adapters"], n, r, dtype=dt, std=r ** -0.5)
        s["scales"] = 0.5 + torch.rand(c["adapters"], generator=g, device="cuda")
        # request lengths: one token each, the rest shared out unevenly
        q = c["requests"]
        if q == c["tokens"]:
            ends = torch.arange(1, q + 1, device="cuda")
        else:
            share = torch.rand(q, generator=g, device="cuda").pow_(4)
            ends = torch.round(torch.cumsum(share, 0) / share.sum() * (c["tokens"] - q)).long()
            ends = ends + torch.arange(1, q + 1, device="cuda")
            ends[-1] = c["tokens"]
        s["segments"] = torch.cat([ends.new_zeros(1), ends]).int()
        # an adapter of each request; about one in eight has none (-1)
        pick = torch.randint(0, c["adapters"], (q,), generator=g, device="cuda")
        none = torch.rand(q, generator=g, device="cuda") < (0.125 if q > 8 else 0.0)
        s["adapters"] = torch.where(none, -1, pick).int()
    return s


# --------------------------------------------------------------------------- the plain forms
def _plain_route(s):
    c, x = s["case"], s["logits"].float()
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    if s["bias"] is not None:
        choice = score + s["bias"]
    else:  # both scores grow with the logit
        choice = x
    if c["groups"] > 1:
        value = choice if s["bias"] is not None else score
        per = value.reshape(x.shape[0], c["groups"], -1)
        best = torch.sort(per, dim=2, descending=True).values[:, :, :c["group_top"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        keep = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        choice = choice.reshape(per.shape).masked_fill(~keep[:, :, None], -math.inf).reshape(x.shape)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :c["top_k"]]
    w = torch.gather(score, 1, ids)
    if c["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    offsets, tokens, where = _plan_of(ids, c["experts"])
    return {"ids": ids.int(), "weights": w * c["scale"], "offsets": offsets, "tokens": tokens,
            "where": where}


def _plain_route_grad(s):
    c, x, ids, dw = s["case"], s["logits"].float(), s["ids"].long(), s["dweights"] * s["case"]["scale"]
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    if c["renormalise"]:
        chosen = torch.gather(score, 1, ids)
        total = chosen.sum(1, keepdim=True)
        dw = (dw - (dw * chosen).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(x).scatter_(1, ids, dw)
    if c["score"] == "sigmoid":
        dx = ds * score * (1.0 - score)
    else:
        dx = score * (ds - (ds * score).sum(1, keepdim=True))
    return {"dlogits": dx.to(s["logits"].dtype)}


def _padded_index(s):
    """Row of each position in an [experts, most] array, a group per expert."""
    off = s["offsets"].long()
    p = torch.arange(s["tokens"].numel(), device=off.device)
    e = torch.bucketize(p, off[1:], right=True)
    return e * s["most"] + p - off[e]


def _spread(rows, at, experts, most):
    out = rows.new_zeros(experts * most, rows.shape[1])
    out[at] = rows
    return out.reshape(experts, most, -1)


def _plain_experts(s):
    c, at = s["case"], _padded_index(s)
    x = _spread(s["x"].float()[s["tokens"].long()], at, c["experts"], s["most"])
    pre = torch.bmm(x, s["w13"].float().transpose(1, 2))
    gate, up = pre[..., :c["inner"]], pre[..., c["inner"]:]
    h = gate / (1.0 + torch.exp(-gate)) * up
    ys = torch.bmm(h, s["w2"].float().transpose(1, 2)).reshape(-1, c["hidden"])[at]
    y = (ys[s["where"].long()] * s["weights"][:, :, None]).sum(1)
    return {"y": y.to(s["x"].dtype)}


def _plain_experts_grad(s):
    c, at, where = s["case"], _padded_index(s), s["where"].long()
    dt = s["dy"].dtype
    dy = s["dy"].float()
    dweights = (s["ys"][where] * dy[:, None, :]).sum(2)
    scaled = s["weights"][:, :, None] * dy[:, None, :]
    dys = torch.empty_like(s["ys"])
    dys[where.reshape(-1)] = scaled.reshape(-1, c["hidden"])
    spread = _spread(dys, at, c["experts"], s["most"])
    inner = _spread(s["inner"].float(), at, c["experts"], s["most"])
    dinner = torch.bmm(spread, s["w2"].float()).reshape(-1, c["inner"])[at]
    dw2 = torch.bmm(spread.transpose(1, 2), inner)
    return {"dweights": dweights, "dys": dys.to(dt), "dinner": dinner.to(dt), "dw2": dw2.to(dt)}


def _plain_lora(s):
    c = s["case"]
    x = s["x"].float()
    y = x @ s["w"].float().T
    token = torch.arange(c["tokens"], device=x.device)
    of = s["adapters"].long()[torch.bucketize(token, s["segments"][1:].long(), right=True)]
    # all adapters at once, each token keeping its own (a product with every adapter's rows)
    t = x @ s["a"].float().reshape(-1, c["k"]).T
    mine = torch.arange(c["adapters"], device=x.device)[None, :] == of[:, None]
    t = t.reshape(c["tokens"], c["adapters"], c["rank"]) * (mine * s["scales"])[:, :, None]
    b = s["b"].float().permute(0, 2, 1).reshape(-1, c["n"])
    return {"y": (y + t.reshape(c["tokens"], -1) @ b).to(s["x"].dtype)}


# --------------------------------------------------------------------------- the library's operators
def _own(s):
    import dense_gemm_sgemm_gb300 as g

    c = s["case"]
    if c["kind"] == "route":
        ids, weights, offsets, tokens, where = g.moe_route(
            s["logits"], c["top_k"], bias=s["bias"], score=c["score"], groups=c["groups"],
            groups_kept=c["kept"], group_top=c["group_top"], renormalise=c["renormalise"],
            scale=c["scale"])
        return {"ids": ids, "weights": weights, "offsets": offsets, "tokens": tokens, "where": where}
    if c["kind"] == "route_grad":
        return {"dlogits": g.moe_route_backward(s["dweights"], s["logits"], s["ids"], score=c["score"],
                                                renormalise=c["renormalise"], scale=c["scale"])}
    if c["kind"] == "experts":
        inner = g.grouped_linear(s["x"], s["w13"], s["offsets"], rows=s["tokens"], gated=True)
        ys = g.grouped_linear(inner, s["w2"], s["offsets"], out_dtype=torch.float32)
        return {"y": g.moe_combine(ys, s["where"], s["weights"], out_dtype=s["x"].dtype)}
    if c["kind"] == "experts_grad":
        dys, dweights = g.moe_combine_backward(s["dy"], s["ys"], s["where"], s["weights"])
        dinner = g.grouped_linear(dys, s["w2"], s["offsets"], opW="N")
        dw2 = g.grouped_weight_grad(dys, s["inner"], s["offsets"], out_dtype=dys.dtype)
        return {"dweights": dweights, "dys": dys, "dinner": dinner, "dw2": dw2}
    return {"y": g.lora_linear(s["x"], s["w"], s["a"], s["b"], s["segments"], s["adapters"],
                               scales=s["scales"])}


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "route_grad": _plain_route_grad, "experts": _plain_experts,
            "experts_grad": _plain_experts_grad, "lora": _plain_lora}[state["case"]["kind"]](state)


# --------------------------------------------------------------------------- floors
def work(case):
    c = case
    t = c["tokens"]
    if c["kind"] == "route":
        b = {"f32": 4, "f16": 2, "bf16": 2}[c["dtype"]]
        e, k = c["experts"], c["top_k"]
        return {"bytes": t * e * b + 4 * e * c["bias"] + t * k * 16 + 4 * (e + 1), "flops": 8 * t * e}
    if c["kind"] == "route_grad":
        b = {"f32": 4, "f16": 2, "bf16": 2}[c["dtype"]]
        return {"bytes": 2 * t * c["experts"] * b + 8 * t * c["top_k"], "flops": 10 * t * c["experts"]}
    if c["kind"] == "lora":
        n, k, r = c["n"], c["k"], c["rank"]
        used = c["adapters"] * (1.0 - (1.0 - 1.0 / c["adapters"]) ** c["requests"])
        return {"bytes": int(2 * (t * k + n * k + t * n + used * r * (n + k))),
                "flops": 2 * t * n * k + 2 * t * r * (n + k)}
    h, i, e = c["hidden"], c["inner"], c["experts"]
    top_k = min(c["top_k"], e)
    rows = t * top_k
    active = e * (1.0 - (1.0 - top_k / e) ** t)  # experts that some token chose, on average
    if c["kind"] == "experts":
        return {"bytes": int(2 * (active * 3 * i * h + 2 * t * h) + 12 * rows),
                "flops": 6 * rows * i * h + 2 * rows * h}
    return {"bytes": int(2 * (active * i * h + e * i * h + t * h + rows * h + 2 * rows * i) + 4 * rows * h
                         + 12 * rows),
            "flops": 4 * rows * i * h + 4 * rows * h}


# --------------------------------------------------------------------------- in 64 bits
def _exact_score(c, x):
    if c["score"] == "sigmoid":
        return torch.sigmoid(x)
    return torch.softmax(x, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    c, kind = case, case["kind"]
    if kind == "route":
        score = _exact_score(c, s["logits"].double())
        value = score if s["bias"] is None else score + s["bias"].double()
        if c["groups"] > 1:
            per = value.reshape(value.shape[0], c["groups"], -1)
            best = torch.topk(per, c["group_top"], dim=2).values.sum(2)
            bar = torch.topk(best, c["kept"], dim=1).values[:, -1:]
            value = torch.where((best >= bar)[:, :, None], per, -math.inf).reshape(value.shape)
        w = torch.gather(score, 1, torch.topk(value, c["top_k"], dim=1).indices)
        if c["renormalise"]:
            w = w / w.sum(1, keepdim=True)
        return {"ids": None, "weights": w * c["scale"], "offsets": None, "tokens": None, "where": None}
    if kind == "route_grad":
        x = s["logits"].double().requires_grad_(True)
        w = torch.gather(_exact_score(c, x), 1, s["ids"].long())
        if c["renormalise"]:
            w = w / w.sum(1, keepdim=True)
        (w * c["scale"]).backward(s["dweights"].double())
        return {"dlogits": x.grad}
    if kind == "lora":
        x = s["x"].double()
        y = x @ s["w"].double().T
        ends, who = s["segments"].tolist(), s["adapters"].tolist()
        for q, a in enumerate(who):
            if a >= 0:
                r = slice(ends[q], ends[q + 1])
                y[r] += s["scales"][a].double() * (x[r] @ s["a"][a].double().T) @ s["b"][a].double().T
        return {"y": y}
    off = s["offsets"].tolist()
    where, weights = s["where"].long(), s["weights"].double()
    if kind == "experts":
        x = s["x"].double()
        ys = x.new_zeros(s["tokens"].numel(), c["hidden"])
        for e in range(c["experts"]):
            r = slice(off[e], off[e + 1])
            pre = x[s["tokens"][r].long()] @ s["w13"][e].double().T
            h = torch.nn.functional.silu(pre[:, :c["inner"]]) * pre[:, c["inner"]:]
            ys[r] = h @ s["w2"][e].double().T
        return {"y": torch.einsum("tk,tkh->th", weights, ys[where])}
    dy = s["dy"].double()
    dys = dy.new_zeros(s["ys"].shape)
    dys[where.reshape(-1)] = torch.einsum("tk,th->tkh", weights, dy).reshape(-1, c["hidden"])
    dinner = dy.new_zeros(s["inner"].shape)
    dw2 = dy.new_zeros(s["w2"].shape)
    for e in range(c["experts"]):
        r = slice(off[e], off[e + 1])
        dinner[r] = dys[r] @ s["w2"][e].double()
        dw2[e] = dys[r].T @ s["inner"][r].double()
    return {"dweights": torch.einsum("th,tkh->tk", dy, s["ys"].double()[where]), "dys": dys,
            "dinner": dinner, "dw2": dw2}
