"""The operators before, inside and after the MoE layer in a training step, as cases that can be timed
and compared: layer norm (with the residual sum) and its gradient, the choice of experts from scores with
a balancing bias and expert groups and its gradient, and the orthogonalised update of the experts' weight
matrices (Muon).

`own` false: plain torch forms, from the formulas. `own` true: the calls a user makes.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}

# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the choice for one decoded token: the launch is all of the time
        dict(name="route-one-token", op="route", T=1, E=128, k=8, groups=1, kept=1, top=1, score="softmax",
             renorm=True, temperature=0.2, scale=1.0, bias=False),
        # a batch over 256 experts in eight groups: sigmoid scores, balancing bias, four groups kept
        dict(name="route-groups", op="route", T=32768, E=256, k=8, groups=8, kept=4, top=2, score="sigmoid",
             renorm=True, temperature=1.0, scale=2.5, bias=True),
        # a small odd layer's gradient: softmax over all experts, weights as they are
        dict(name="route-grad-odd", op="route_grad", T=777, E=45, k=3, groups=1, kept=1, top=1, score="softmax",
             renorm=False, temperature=0.7, scale=1.0, bias=False),
        # the gradient of the batch over 256 experts
        dict(name="route-grad-groups", op="route_grad", T=32768, E=256, k=8, groups=8, kept=4, top=2,
             score="sigmoid", renorm=True, temperature=1.0, scale=2.5, bias=True),
        # a small fp32 model with odd rows
        dict(name="norm-small-fp32", op="norm", T=777, d=37, dtype="f32", params="f32", residual=False),
        # the hybrid layer's batch: residual sum and norm of it in one pass
        dict(name="norm-batch", op="norm", T=16384, d=1024, dtype="bf16", params="f32", residual=True),
        # odd fp32 rows, gradients of gain and bias
        dict(name="norm-grad-odd-fp32", op="norm_grad", T=2047, d=1023, dtype="f32", params="f32", residual=False),
        # the widest layer's batch, with the gradient that comes past the layer added
        dict(name="norm-grad-wide", op="norm_grad", T=32768, d=2048, dtype="bf16", params="f32", residual=True),
        # the gate's weight, fp32: few small matrix products, one after another
        dict(name="ortho-gate-fp32", op="ortho", count=1, rows=128, cols=1024, dtype="f32"),
        # all of the hybrid layer's second expert weights, wide matrices
        dict(name="ortho-e128", op="ortho", count=128, rows=1024, cols=4096, dtype="bf16"),
        # a step on a small fp32 layer's experts, odd sizes
        dict(name="muon-small-odd", op="muon", count=5, rows=45, cols=37, dtype="f32", grad="f32", nesterov=True),
        # a step on the 16 experts' first weights, tall matrices
        dict(name="muon-e16", op="muon", count=16, rows=4096, cols=1024, dtype="bf16", grad="bf16", nesterov=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "norm", "norm_grad", "ortho", "muon"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("route", "route_grad"):
        c = dict(op=op, T=_log(rng, 1, 32768), score=rng.choice(["softmax", "sigmoid"]),
                 renorm=rng.random() < 0.7, temperature=rng.choice([1.0, 0.7, 0.2]), scale=rng.choice([1.0, 2.5]),
                 bias=rng.random() < 0.6)
        if rng.random() < 0.5:
            c["groups"] = rng.choice([2, 4, 5, 8])
            c["E"] = c["groups"] * rng.randint(4, 256 // c["groups"])
            c["kept"], c["top"] = rng.randint(1, c["groups"] - 1), rng.choice([1, 2])
        else:
            c.update(groups=1, kept=1, top=1, E=rng.randint(4, 256))
        c["k"] = rng.randint(1, min(8, c["E"] // c["groups"] * c["kept"] // 2))
        c["renorm"] = c["renorm"] and c["k"] > 1       # a single weight is not divided by itself
        return c
    if op in ("norm", "norm_grad"):
        d = _log(rng, 33, 8200)
        if rng.random() < 0.6:
            d = max(64, d // 64 * 64)
        return dict(op=op, T=_log(rng, 1, min(32768, 60_000_000 // d)), d=d, dtype=dtype,
                    params=rng.choice([dtype, "f32"]), residual=rng.random() < 0.5)
    # matrices of a layer: the products of one stay within the largest listed case's
    rows, cols = _log(rng, 24, 4200), _log(rng, 24, 4200)
    if rng.random() < 0.6:
        rows, cols = max(32, rows // 32 * 32), max(32, cols // 32 * 32)
    one = min(rows, cols) ** 2 * max(rows, cols)
    c = dict(op=op, count=min(_log(rng, 1, 64), max(1, 16 * 1024 * 1024 * 4096 // one)), rows=rows, cols=cols,
             dtype=dtype)
    if op == "muon":
        c.update(grad=rng.choice([dtype, "f32"]), nesterov=rng.random() < 0.7)
    return c


# ------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(shape, dtype, g, std=1.0):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    return x.normal_(0.0, std, generator=g)


# Added to the sum that weights are divided by: sigmoids can all be zero in 32 bits.
TINY = {"softmax": 0.0, "sigmoid": 1e-20}
# Two choices whose scores differ by less are both right where scores are rounded to 32 bits.
MARGIN = 4e-6


def _choice64(z, bias, c):
    """Experts by score in 64 bits: chosen [T, k], scores [T, E], and which rows have no two
    near-equal scores or groups where the choice is made."""
    T, E, G = z.shape[0], c["E"], c["groups"]
    x = z.double() / c["temperature"]
    s = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
    v = s if bias is None else s + bias.double()
    clear = torch.ones(T, dtype=torch.bool, device=z.device)

    def apart(hi, lo):
        gap = hi - lo
        return gap > MARGIN * (1 if bias is not None else hi.abs().clamp(max=1))

    if c["kept"] < G:
        by = v.view(T, G, E // G)
        worth = by.topk(min(c["top"], E // G), 2).values.sum(2)
        top = worth.sort(1, descending=True)
        clear &= apart(top.values[:, c["kept"] - 1], top.values[:, c["kept"]])
        out = torch.ones(T, G, dtype=torch.bool, device=z.device).scatter_(1, top.indices[:, :c["kept"]], False)
        v = by.masked_fill(out[:, :, None], -math.inf).view(T, E)
    top = v.topk(min(c["k"] + 1, E), 1)
    if top.values.shape[1] > 1:
        near = apart(top.values[:, :-1], top.values[:, 1:])
        clear &= (near | torch.isinf(top.values[:, 1:])).all(1)
    return top.indices[:, :c["k"]], s, clear


def _logits(c, g):
    """Gate outputs: normal around a popularity of the expert. Rows with two near-equal scores are
    drawn again, for there either choice is right."""
    T, E = c["T"], c["E"]
    popular = _randn((E,), torch.float32, g, 0.3)
    bias = _randn((E,), torch.float32, g, 0.02) if c["bias"] else None
    z = _randn((T, E), torch.float32, g, 0.64) + popular
    for _ in range(40):
        idx, _, clear = _choice64(z, bias, c)
        rows = (~clear).nonzero()[:, 0]
        if rows.numel() == 0:
            break
        z[rows] = _randn((rows.numel(), E), torch.float32, g, 0.64) + popular
    return z, bias, idx.to(torch.int32)


def _matrices(shape, dtype, g, size):
    """Gradients of weight matrices: a few strong directions over noise."""
    n, rows, cols = shape
    r = min(8, rows, cols)
    left, right = _randn((n, rows, r), torch.float32, g), _randn((n, r, cols), torch.float32, g)
    fall = torch.logspace(0, -2, r, device="cuda")
    x = _randn(shape, torch.float32, g, size)
    return x.baddbmm_(left * (fall * size), right, beta=0.5).to(dtype)


STEPS, COEF = 5, (3.4445, -4.7750, 2.0315)
HYPER = dict(lr=0.02, momentum=0.95, weight_decay=0.1)


def _muon_scale(c):
    return 0.2 * math.sqrt(max(c["rows"], c["cols"]))


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": dict(c)}
    if c["op"] in ("route", "route_grad"):
        s["z"], s["bias"], idx = _logits(c, g)
        if c["op"] == "route":
            s["idx"], s["w"] = torch.empty_like(idx), torch.empty(idx.shape, device="cuda")
            s["counts"] = torch.empty(c["E"], dtype=torch.int32, device="cuda")
            s["balance"] = torch.empty(1, device="cuda")
        else:
            s["idx"], s["dw"] = idx, _randn(idx.shape, torch.float32, g, 0.05)
            s["dz"] = torch.empty_like(s["z"])
    elif c["op"] in ("norm", "norm_grad"):
        T, d, dt, pt = c["T"], c["d"], DT[c["dtype"]], DT[c["params"]]
        # activations: rows of different size and offset, a few columns far larger than the rest
        size = torch.empty((T, 1), device="cuda").log_normal_(0.0, 0.5, generator=g)
        heavy = 1 + 8 * (torch.rand(d, generator=g, device="cuda") < 0.01)
        x = _randn((T, d), torch.float32, g).mul_(heavy).add_(_randn((T, 1), torch.float32, g, 0.3)).mul_(size)
        s["gain"] = (1 + _randn((d,), torch.float32, g, 0.1)).to(pt)
        s["x"] = x.to(dt)
        if c["op"] == "norm":
            s["bias"] = _randn((d,), torch.float32, g, 0.1).to(pt)
            s["r"] = _randn((T, d), dt, g) if c["residual"] else None
            s["sum"] = torch.empty_like(s["x"]) if c["residual"] else None
            s["y"] = torch.empty_like(s["x"])
            s["mean"], s["rstd"] = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        else:
            # statistics as the forward pass leaves them
            x = s["x"].double()
            mean = x.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = ((x - mean[:, None]).square_().mean(1) + EPS).rsqrt().float()
            s["dy"] = _randn((T, d), dt, g, 0.01)
            s["dsum"] = _randn((T, d), dt, g, 0.01) if c["residual"] else None
            s["dx"] = torch.empty_like(s["dy"])
            s["dgain"], s["dbias"] = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    else:
        shape, dt = (c["count"], c["rows"], c["cols"]), DT[c["dtype"]]
        s["g"] = _matrices(shape, DT[c.get("grad", c["dtype"])], g, 1e-3)
        if c["op"] == "ortho":
            s["o"] = torch.empty(shape, dtype=dt, device="cuda")
        else:
            s["p"] = _randn(shape, dt, g, 0.02)
            s["m"] = _matrices(shape, torch.float32, g, 5e-3)
    return s


EPS = 1e-5

# ------------------------------------------------------------------------------------ the passes

def run(state):
    return {"route": _route, "route_grad": _route_grad, "norm": _norm, "norm_grad": _norm_grad, "ortho": _ortho,
            "muon": _muon}[state["case"]["op"]](state)


def _score_config(s, c):
    import token_routing_gb300 as moe
    s["cfg"] = moe.make_score_config(c["T"], c["E"], c["k"], score=c["score"], groups=c["groups"],
                                     groups_kept=c["kept"], group_top=c["top"], renormalise=c["renorm"],
                                     temperature=c["temperature"], scale=c["scale"])
    return moe


def _route(s):
    c = s["case"]
    if own:
        import token_routing_gb300 as moe
        if "cfg" not in s:
            _score_config(s, c)
            s["ws"] = torch.empty(moe.route_scores_workspace_bytes(s["cfg"]), dtype=torch.uint8, device="cuda")
        moe.route_scores(s["cfg"], s["z"], s["bias"], s["idx"], s["w"], s["counts"], s["balance"], s["ws"])
        return {k: s[k] for k in ("idx", "w", "counts", "balance")}
    T, E, G = c["T"], c["E"], c["groups"]
    score = _scores(s["z"], c)
    v = score if s["bias"] is None else score + s["bias"]
    if c["kept"] < G:
        by = v.view(T, G, E // G)
        first = by.amax(2)
        worth = first
        if c["top"] == 2 and E // G > 1:
            at = by.argmax(2, keepdim=True)
            worth = first + by.scatter(2, at, -math.inf).amax(2)
        order = worth.sort(dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device="cuda").scatter_(1, order, True)
        v = by.masked_fill(~keep[:, :, None], -math.inf).view(T, E)
    idx = v.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = score.gather(1, idx)
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + TINY[c["score"]])
    counts = torch.zeros(E, dtype=torch.int64, device="cuda").index_add_(0, idx.reshape(-1),
                                                                         torch.ones_like(idx.reshape(-1)))
    balance = (counts.double() - T * c["k"] / E).square().mean().float().reshape(1)
    return {"idx": idx.to(torch.int32), "w": w * c["scale"], "counts": counts.to(torch.int32), "balance": balance}


def _scores(z, c):
    x = z / c["temperature"]
    if c["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _route_grad(s):
    c = s["case"]
    if own:
        import token_routing_gb300 as moe
        if "cfg" not in s:
            _score_config(s, c)
        moe.route_scores_backward(s["cfg"], s["z"], s["idx"], s["dw"], s["dz"])
        return s["dz"]
    idx, dw = s["idx"].long(), s["dw"]
    score = _scores(s["z"], c)
    picked = score.gather(1, idx)
    if c["renorm"]:
        # through the division by the sum; by differences, since one weight can be nearly all of it
        total = picked.sum(1, keepdim=True) + TINY[c["score"]]
        share = picked / total
        g = (share[:, None, :] * (dw[:, :, None] - dw[:, None, :])).sum(2) + dw * (TINY[c["score"]] / total)
        g = g * (c["scale"] / total)
    else:
        g = dw * c["scale"]
    if c["score"] == "sigmoid":
        d = g * picked / (1 + torch.exp(s["z"].gather(1, idx) / c["temperature"]))
    elif c["renorm"]:
        d = g * picked
    else:
        dense = torch.zeros_like(score).scatter_(1, idx, g)
        return score * (dense - (picked * g).sum(1, keepdim=True)) / c["temperature"]
    return torch.zeros_like(score).scatter_(1, idx, d / c["temperature"])


def _norm(s):
    c = s["case"]
    if own:
        import token_routing_gb300 as moe
        if "cfg" not in s:
            s["cfg"] = moe.make_norm_config(c["T"], c["d"], eps=EPS, dtype=c["dtype"], param_dtype=c["params"])
        moe.layer_norm(s["cfg"], s["x"], s["gain"], s["bias"], s["y"], residual=s["r"], total=s["sum"],
                       mean=s["mean"], rstd=s["rstd"])
        return {k: s[k] for k in ("y", "sum", "mean", "rstd") if s[k] is not None}
    x = s["x"].float()
    if s["r"] is not None:
        x = x + s["r"].float()
    mean = x.mean(1, keepdim=True)
    off = x - mean
    rstd = 1 / torch.sqrt((off * off).mean(1, keepdim=True) + EPS)
    y = off * rstd * s["gain"].float() + s["bias"].float()
    out = {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if s["r"] is not None:
        out["sum"] = x.to(s["x"].dtype)
    return out


def _norm_grad(s):
    c = s["case"]
    if own:
        import token_routing_gb300 as moe
        if "cfg" not in s:
            s["cfg"] = moe.make_norm_config(c["T"], c["d"], eps=EPS, dtype=c["dtype"], param_dtype=c["params"])
            s["ws"] = torch.empty(moe.norm_workspace_bytes(s["cfg"]), dtype=torch.uint8, device="cuda")
        moe.layer_norm_backward(s["cfg"], s["dy"], s["x"], s["gain"], s["mean"], s["rstd"], s["dx"], s["dgain"],
                                s["dbias"], s["ws"], dtotal=s["dsum"])
        return {k: s[k] for k in ("dx", "dgain", "dbias")}
    dy, hat = s["dy"].float(), (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["gain"].float()
    dx = (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(s["dy"].dtype), "dgain": (dy * hat).sum(0, dtype=torch.float64).float(),
            "dbias": dy.sum(0, dtype=torch.float64).float()}


def _orthogonal(u):
    """Newton-Schulz: the singular values of each matrix go near one, its directions stay."""
    a, b, c = COEF
    tall = u.shape[1] > u.shape[2]
    x = u.transpose(1, 2) if tall else u
    x = x / (x.square().sum((1, 2), keepdim=True, dtype=torch.float64).sqrt().float() + 1e-7)
    for _ in range(STEPS):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.transpose(1, 2) if tall else x


def _ortho(s):
    c = s["case"]
    if own:
        import token_routing_gb300 as moe
        if "cfg" not in s:
            s["cfg"] = moe.make_muon_config(c["count"], c["rows"], c["cols"], dtype=c["dtype"], steps=STEPS, coef=COEF)
            s["ws"] = torch.empty(moe.muon_workspace_bytes(s["cfg"]), dtype=torch.uint8, device="cuda")
        moe.orthogonalize(s["cfg"], s["g"], s["o"], s["ws"])
        return s["o"]
    return _orthogonal(s["g"].float()).to(s["g"].dtype)


def _muon(s):
    c, h = s["case"], HYPER
    if own:
        import token_routing_gb300 as moe
        if "opt" not in s:
            s["opt"] = moe.Muon([dict(p=s["p"], g=s["g"], m=s["m"], scale=_muon_scale(c))], lr=h["lr"],
                                momentum=h["momentum"], weight_decay=h["weight_decay"], nesterov=c["nesterov"],
                                steps=STEPS, coef=COEF)
        s["opt"].step()
        return {"p": s["p"], "m": s["m"]}
    g = s["g"].float()
    s["m"].copy_(h["momentum"] * s["m"] + g)
    u = g + h["momentum"] * s["m"] if c["nesterov"] else s["m"]
    s["p"].copy_(s["p"].float() * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * _muon_scale(c) * _orthogonal(u))
    return {"p": s["p"], "m": s["m"]}


# ------------------------------------------------------------------------------------ the least work

def work(case):
    c = case
    if c["op"] == "route":
        return {"bytes": 4 * c["T"] * (c["E"] + 2 * c["k"]) + 8 * c["E"], "flops": 8 * c["T"] * c["E"]}
    if c["op"] == "route_grad":
        # where only chosen experts have a gradient, only their logits are read
        read = c["E"] if c["score"] == "softmax" and not c["renorm"] else c["k"]
        return {"bytes": 4 * c["T"] * (c["E"] + read + 2 * c["k"]), "flops": 8 * c["T"] * read}
    if c["op"] in ("norm", "norm_grad"):
        n, es, ps = c["T"] * c["d"], ES[c["dtype"]], ES[c["params"]]
        if c["op"] == "norm":
            return {"bytes": n * es * (4 if c["residual"] else 2) + 8 * c["T"] + 2 * c["d"] * ps, "flops": 8 * n}
        return {"bytes": n * es * (4 if c["residual"] else 3) + 8 * c["T"] + c["d"] * (ps + 8), "flops": 14 * n}
    m, n = sorted((c["rows"], c["cols"]))
    # a step: X X' and its square are symmetric, so half of each is enough; and one full product
    flops = c["count"] * STEPS * (m * m * n + m * m * m + 2 * m * m * n)
    size = c["count"] * m * n
    if c["op"] == "ortho":
        return {"bytes": 2 * size * ES[c["dtype"]], "flops": flops}
    return {"bytes": size * (2 * ES[c["dtype"]] + ES[c["grad"]] + 8), "flops": flops}


# ------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s, c = prepare(case, seed), case
    return {"route": _exact_route, "route_grad": _exact_route_grad, "norm": _exact_norm, "norm_grad": _exact_norm_grad,
            "ortho": _exact_ortho, "muon": _exact_muon}[c["op"]](s, c)


def _exact_route(s, c):
    idx, score, _ = _choice64(s["z"], s["bias"], c)
    w = torch.take_along_dim(score, idx, 1)
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + TINY[c["score"]])
    counts = torch.bincount(idx.reshape(-1), minlength=c["E"])
    balance = ((counts.double() - counts.double().mean()) ** 2).mean().reshape(1)
    return {"idx": idx.to(torch.int32), "w": w * c["scale"], "counts": counts.to(torch.int32), "balance": balance}


def _exact_route_grad(s, c):
    """By automatic differentiation of the weights in 64 bits."""
    z = s["z"].double().requires_grad_(True)
    x = z / c["temperature"]
    score = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
    w = torch.take_along_dim(score, s["idx"].long(), 1)
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + TINY[c["score"]])
    (dz,) = torch.autograd.grad((c["scale"] * w * s["dw"].double()).sum(), z)
    return dz


def _exact_norm(s, c):
    x = s["x"].double()
    if c["residual"]:
        x = x + s["r"].double()
    mean, var = x.mean(1), x.var(1, unbiased=False)
    rstd = (var + EPS) ** -0.5
    y = (x - mean[:, None]) * rstd[:, None] * s["gain"].double() + s["bias"].double()
    out = {"y": y, "mean": mean, "rstd": rstd}
    if c["residual"]:
        out["sum"] = x
    return out


def _exact_norm_grad(s, c):
    """The Jacobian as a projection: dx = rstd (I - 1 1'/d - h h'/d) (gain dy), on the saved statistics."""
    dy, r = s["dy"].double(), s["rstd"].double()[:, None]
    h = (s["x"].double() - s["mean"].double()[:, None]) * r
    v = dy * s["gain"].double()
    d = c["d"]
    dx = r * (v - v.sum(1, keepdim=True) / d - h * ((h * v).sum(1, keepdim=True) / d))
    if c["residual"]:
        dx = dx + s["dsum"].double()
    return {"dx": dx, "dgain": torch.einsum("td,td->d", dy, h), "dbias": dy.sum(0)}


def _exact_polar(u):
    """The odd polynomial on the singular values, by way of the small Gram matrix: every iterate is
    q(A) u with A = u u' (or u' u), and q of A commutes with A."""
    a, b, c = COEF
    tall = u.shape[0] > u.shape[1]
    u = u / (torch.linalg.matrix_norm(u) + 1e-7)
    A = u.T @ u if tall else u @ u.T
    eye = torch.eye(A.shape[0], dtype=torch.float64, device="cuda")
    q = eye
    for k in range(STEPS):
        f = a * eye + b * A + c * (A @ A)
        q = f @ q
        if k + 1 < STEPS:
            A = f @ A @ f
    return u @ q if tall else q @ u


def _exact_ortho(s, c):
    out = torch.empty(s["g"].shape, dtype=torch.float64, device="cuda")
    for i in range(c["count"]):
        out[i] = _exact_polar(s["g"][i].double())
    return out


def _exact_muon(s, c):
    mu, lr, decay = HYPER["momentum"], HYPER["lr"], HYPER["weight_decay"]
    g = s["g"].double()
    m = mu * s["m"].double() + g
    u = g + mu * m if c["nesterov"] else m
    p = s["p"].double() * (1 - lr * decay)
    for i in range(c["count"]):
        p[i] -= lr * _muon_scale(c) * _exact_polar(u[i])
    return {"p": p, "m": m}
