"""The operators around the MoE layer in a training step, as cases that can be timed and compared:
the embedding lookup that makes the layer's input and the gradient that takes its dx, the clipped
policy loss with a KL term on the logits, and the AdamW step over all of the weights.

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
        # one decoded token's row: the launch is all of the time
        dict(name="embed-one-token", op="embed", T=1, V=32000, d=1024, dtype="bf16", scale=1.0),
        # the batch of the hybrid top-8 layer, scaled by sqrt(d)
        dict(name="embed-batch", op="embed", T=16384, V=131072, d=1024, dtype="bf16", scale=32.0),
        # a small fp32 model: odd row length, ragged batch, whole gradient written
        dict(name="embed-grad-small-fp32", op="embed_grad", T=777, V=1009, d=37, dtype="f32", grad="f32",
             scale=1.0, accumulate=False, pad=0),
        # the hybrid layer's batch into a large vocabulary's bf16 gradient, written whole
        dict(name="embed-grad-batch", op="embed_grad", T=16384, V=131072, d=1024, dtype="bf16", grad="bf16",
             scale=32.0, accumulate=False, pad=-1),
        # tied weights: the Zipf layer's width, added into the fp32 gradient that the output head has begun
        dict(name="embed-grad-tied", op="embed_grad", T=32768, V=50021, d=2048, dtype="bf16", grad="f32",
             scale=1.0, accumulate=True, pad=1),
        # log-probabilities of a few sampled tokens, as a server gives them: one row for many SMs
        dict(name="logp-few", op="logp", T=4, V=131072, dtype="bf16", temperature=0.7),
        # the reference model's log-probabilities of a batch, fp32 logits
        dict(name="logp-batch-fp32", op="logp", T=4096, V=32000, dtype="f32", temperature=1.0),
        # an odd vocabulary: rows start at every alignment
        dict(name="policy-odd-vocab", op="policy", T=2048, V=50021, dtype="bf16", temperature=1.0, kl=0.04,
             masked=0.25),
        # a long batch of rollouts at a large vocabulary, prompts masked
        dict(name="policy-large", op="policy", T=8192, V=131072, dtype="bf16", temperature=1.0, kl=0.02,
             masked=0.2),
        # many small tensors (norms, biases, narrow gates) in one call: launches count
        dict(name="adamw-many-small", op="adamw", layers=24, E=5, d=37, f=45, V=0, dtype="f32", bits=32,
             master=False),
        # the 16-expert layer with its embedding: bf16 weights, fp32 masters and states
        dict(name="adamw-e16", op="adamw", layers=1, E=16, d=1024, f=4096, V=32000, dtype="bf16", bits=32,
             master=True),
        # the hybrid layer's 128 experts with states in 8 bits
        dict(name="adamw-e128-8bit", op="adamw", layers=1, E=128, d=1024, f=4096, V=32000, dtype="bf16", bits=8,
             master=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "embed_grad", "logp", "policy", "policy", "adamw", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("embed", "embed_grad"):
        c = dict(op=op, T=_log(rng, 1, 32768), V=_log(rng, 500, 131072), d=_log(rng, 33, 2100), dtype=dtype,
                 scale=rng.choice([1.0, 8.0, 0.5]))
        if rng.random() < 0.6:
            c["d"] = max(64, c["d"] // 64 * 64)
        if op == "embed_grad":
            c.update(grad=rng.choice([dtype, "f32"]), accumulate=rng.random() < 0.5,
                     pad=rng.choice([-1, 0, c["V"] - 1]))
        return c
    if op in ("logp", "policy"):
        V = _log(rng, 500, 140000)
        if rng.random() < 0.5:
            V = V // 64 * 64 + 64
        c = dict(op=op, T=_log(rng, 1, max(2, min(16384, 500_000_000 // V))), V=V, dtype=dtype,
                 temperature=rng.choice([1.0, 0.7, 1.3]))
        if op == "policy":
            c.update(kl=rng.choice([0.0, 0.01, 0.1]), masked=rng.choice([0.0, 0.25, 0.75]))
        return c
    c = dict(op=op, layers=1, E=rng.randint(1, 32), d=_log(rng, 33, 1100), f=_log(rng, 33, 4200),
             V=rng.choice([0, _log(rng, 500, 32000)]), dtype=dtype, bits=rng.choice([8, 32]),
             master=dtype == "bf16" and rng.random() < 0.7)
    if rng.random() < 0.4:
        c.update(layers=rng.randint(2, 40), E=rng.randint(1, 8), d=rng.randint(33, 200), f=rng.randint(33, 300))
    return c


# ------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _zipf(V):
    """Token frequencies: p(rank) ~ 1 / (rank + 2.7), the usual law for words."""
    p = 1.0 / (torch.arange(V, dtype=torch.float64) + 2.7)
    return p / p.sum()


def _tokens(T, V, g):
    cdf = torch.cumsum(_zipf(V), 0).cuda()
    rank = torch.searchsorted(cdf, torch.rand(T, generator=g, device="cuda", dtype=torch.float64)).clamp_(max=V - 1)
    order = torch.randperm(V, generator=g, device="cuda")
    return order[rank].to(torch.int32)


def _randn(shape, dtype, g, std=1.0):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    return x.normal_(0.0, std, generator=g)


def _tensors(c):
    """The weights of `layers` MoE layers and an embedding table, in the layer's own types:
    (elements, weight is fp32, gradient is fp32, decayed)."""
    E, d, f, one = c["E"], c["d"], c["f"], c["dtype"] == "f32"
    layer = [(E * d, one, True, True),            # Wg, dWg fp32
             (E, True, True, False),              # bg
             (E * f * d, one, one, True),         # W1
             (E * f, one, True, False),           # b1, db1 fp32
             (E * d * f, one, one, True),         # W2
             (E * d, one, True, False)]           # b2
    table = [(c["V"] * d, one, one, True)] if c["V"] else []
    return table + layer * c["layers"]


def _carve(sizes, dtype, unit=64):
    """One buffer and its views, each on a boundary of `unit` elements."""
    at = [0]
    for n in sizes:
        at.append(at[-1] + (n + unit - 1) // unit * unit)
    flat = torch.zeros(at[-1], dtype=dtype, device="cuda")
    return flat, [flat[a:a + n] for a, n in zip(at, sizes)]


HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8)
DECAY = 0.1
BLOCK = 256  # elements to a scale of the 8-bit states


def _mean_before(grad, g):
    """First and second moments as earlier steps leave them: of the gradient's size, row by row."""
    return torch.empty(grad.shape, device="cuda").normal_(0.0, 0.5, generator=g).mul_(grad.float().abs_()).add_(
        grad.float(), alpha=0.1)


def _root_before(grad, g):
    return torch.empty(grad.shape, device="cuda").log_normal_(0.0, 0.5, generator=g).mul_(grad.float().abs_())


def _prepare_adamw(c, g):
    spec = _tensors(c)
    s = {"flat": {}}
    views = {}
    for key, want in (("p16", [n for n, p32, _, _ in spec if not p32]), ("p32", [n for n, p32, _, _ in spec if p32]),
                      ("g16", [n for n, _, g32, _ in spec if not g32]), ("g32", [n for n, _, g32, _ in spec if g32])):
        dt = torch.bfloat16 if key.endswith("16") else torch.float32
        flat, v = _carve(want, dt)
        s["flat"][key], views[key] = flat, iter(v)
    s["p"] = [next(views["p32" if p32 else "p16"]) for _, p32, _, _ in spec]
    s["g"] = [next(views["g32" if g32 else "g16"]) for _, _, g32, _ in spec]
    s["decay"] = [DECAY if dec else 0.0 for _, _, _, dec in spec]
    for k in ("p16", "p32"):
        s["flat"][k].normal_(0.0, 0.02, generator=g)
    # gradients of very different sizes from tensor to tensor and, within one, from row to row
    for t in s["g"]:
        t.normal_(0.0, 1e-3, generator=g)
        rows = t[:t.numel() // 64 * 64].view(-1, 64)
        rows.mul_(torch.empty((rows.shape[0], 1), device="cuda").log_normal_(0.0, 1.5, generator=g).to(t.dtype))
    if c["master"]:
        s["flat"]["w"], s["w"] = _carve([t.numel() if t.dtype == torch.bfloat16 else 0 for t in s["p"]], torch.float32)
        s["w"] = [w if w.numel() else None for w in s["w"]]
        for p, w in zip(s["p"], s["w"]):
            if w is not None:
                w.copy_(p)
    else:
        s["w"] = [None] * len(s["p"])
    sizes = [t.numel() for t in s["p"]]
    if c["bits"] == 32:
        s["flat"]["m"], s["m"] = _carve(sizes, torch.float32)
        s["flat"]["v"], s["v"] = _carve(sizes, torch.float32)
        s["ms"] = s["vs"] = [None] * len(sizes)
        for gr, m, v in zip(s["g"], s["m"], s["v"]):
            m.copy_(_mean_before(gr, g))
            v.copy_(_root_before(gr, g).square_())
    else:
        s["flat"]["m"], s["m"] = _carve(sizes, torch.float8_e4m3fn)
        s["flat"]["v"], s["v"] = _carve(sizes, torch.float8_e4m3fn)
        blocks = [(n + BLOCK - 1) // BLOCK for n in sizes]
        s["flat"]["ms"], s["ms"] = _carve(blocks, torch.float32)
        s["flat"]["vs"], s["vs"] = _carve(blocks, torch.float32)
        half = torch.full((1,), 0x80000, dtype=torch.int64, device="cuda")
        for gr, m, v, ms, vs in zip(s["g"], s["m"], s["v"], s["ms"], s["vs"]):
            _quantise(_mean_before(gr, g), m, ms, half, False)
            _quantise(_root_before(gr, g), v, vs, half, True)
    s["step"] = 20
    return s


def prepare(case, seed):
    c, g = case, _gen(seed)
    dt = DT.get(c.get("dtype"))
    if c["op"] == "adamw":
        s = _prepare_adamw(c, g)
    elif c["op"] == "embed":
        s = dict(ids=_tokens(c["T"], c["V"], g), W=_randn((c["V"], c["d"]), dt, g, 0.02),
                 y=torch.empty((c["T"], c["d"]), dtype=dt, device="cuda"))
    elif c["op"] == "embed_grad":
        s = dict(ids=_tokens(c["T"], c["V"], g), dy=_randn((c["T"], c["d"]), dt, g, 0.01))
        s["dW"] = _randn((c["V"], c["d"]), DT[c["grad"]], g, 0.01)
    else:
        # logits as a head gives them: a spread of a few units; half of the tokens' targets are likely ones
        T, V, tau = c["T"], c["V"], c["temperature"]
        z = _randn((T, V), dt, g, 2.5)
        target = torch.randint(0, V, (T,), generator=g, device="cuda")
        likely = torch.rand(T, generator=g, device="cuda") < 0.5
        z[torch.arange(T, device="cuda"), target] += (likely * 12.0).to(dt)
        s = dict(z=z, target=target.to(torch.int32), logp=torch.empty(T, dtype=torch.float32, device="cuda"))
        if c["op"] == "policy":
            lp = _logp_rows(z, target, tau)
            # the log ratio to the rollout's policy. One within rounding of a clipping border has two
            # right gradients, so none is put there.
            lr = torch.randn(T, generator=g, device="cuda", dtype=torch.float64) * 0.15
            for border in (math.log(0.8), math.log(1.2)):
                lr = torch.where((lr - border).abs() < 1e-4, lr + 3e-4, lr)
            s["old"] = (lp - lr).float()
            s["ref"] = (lp + 0.1 * torch.randn(T, generator=g, device="cuda", dtype=torch.float64)).float()
            s["adv"] = torch.randn(T, generator=g, device="cuda")
            kept = torch.rand(T, generator=g, device="cuda") >= c["masked"]
            if T > 2:
                kept[T // 2] = True
            s["weight"] = kept.float() / kept.sum().clamp(min=1)
            s["loss"] = torch.empty(1, dtype=torch.float32, device="cuda")
            s["dz"] = torch.empty_like(z)
    s["case"] = dict(c)
    return s


def _logp_rows(z, target, tau, rows=1024):
    """log softmax(z / tau)[target], a thousand rows at a time, in 64 bits."""
    got = [_logp64(z[a:a + rows], target[a:a + rows], tau) for a in range(0, z.shape[0], rows)]
    return torch.cat(got)


def _logp64(z, target, tau):
    z = z.double() / tau
    return z.gather(1, target.long()[:, None])[:, 0] - torch.logsumexp(z, 1)


# ------------------------------------------------------------------------------------ the passes

def run(state):
    return {"embed": _embed, "embed_grad": _embed_grad, "logp": _logp, "policy": _policy,
            "adamw": _adamw}[state["case"]["op"]](state)


def _embed(s):
    c = s["case"]
    if own:
        import token_routing_gb300 as moe
        if "cfg" not in s:
            s["cfg"] = moe.make_embed_config(c["T"], c["V"], c["d"], scale=c["scale"], dtype=c["dtype"])
        moe.embed(s["cfg"], s["ids"], s["W"], s["y"])
        return s["y"]
    return (s["W"][s["ids"]].float() * c["scale"]).to(s["W"].dtype)


def _embed_grad(s):
    c = s["case"]
    if own:
        import token_routing_gb300 as moe
        if "cfg" not in s:
            s["cfg"] = moe.make_embed_config(c["T"], c["V"], c["d"], scale=c["scale"], dtype=c["dtype"],
                                             grad_dtype=c["grad"], accumulate=c["accumulate"], padding_id=c["pad"])
            s["ws"] = torch.empty(moe.embed_workspace_bytes(s["cfg"]), dtype=torch.uint8, device="cuda")
        moe.embed_backward(s["cfg"], s["ids"], s["dy"], s["dW"], s["ws"])
        return s["dW"]
    ids = s["ids"].long()
    rows = s["dy"].float() * c["scale"]
    if c["pad"] >= 0:
        rows = rows * (ids != c["pad"])[:, None]
    if c["accumulate"] and s["dW"].dtype == torch.float32:
        return s["dW"].index_add_(0, ids, rows)
    total = torch.zeros(c["V"], c["d"], dtype=torch.float32, device="cuda").index_add_(0, ids, rows)
    if c["accumulate"]:
        return s["dW"].copy_(total + s["dW"].float())
    return total.to(s["dW"].dtype)


def _logp(s):
    c = s["case"]
    if own:
        import token_routing_gb300 as moe
        if "cfg" not in s:
            s["cfg"] = moe.make_policy_config(c["T"], c["V"], dtype=c["dtype"], temperature=c["temperature"])
        moe.token_logp(s["cfg"], s["z"], s["target"], s["logp"])
        return s["logp"]
    z = s["z"].float() / c["temperature"]
    top = z.amax(1, keepdim=True)
    total = torch.exp(z - top).sum(1)
    return z.gather(1, s["target"].long()[:, None])[:, 0] - top[:, 0] - torch.log(total)


CLIP = 0.2


def _policy(s):
    c = s["case"]
    if own:
        import token_routing_gb300 as moe
        if "cfg" not in s:
            s["cfg"] = moe.make_policy_config(c["T"], c["V"], dtype=c["dtype"], temperature=c["temperature"],
                                              clip_low=CLIP, clip_high=CLIP, kl_weight=c["kl"])
            s["ws"] = torch.empty(moe.policy_workspace_bytes(s["cfg"]), dtype=torch.uint8, device="cuda")
        moe.policy_loss(s["cfg"], s["z"], s["target"], s["adv"], s["old"], s["ref"], s["weight"], s["logp"],
                        s["loss"], s["dz"], s["ws"])
        return {"logp": s["logp"], "loss": s["loss"], "dlogits": s["dz"]}
    target, tau = s["target"].long()[:, None], c["temperature"]
    z = s["z"].float() / tau
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    logp = (z.gather(1, target) - top - torch.log(total))[:, 0]
    kept = s["weight"] != 0
    ratio = torch.exp(logp - s["old"])
    clipped = ratio.clamp(1 - CLIP, 1 + CLIP)
    gain = torch.minimum(ratio * s["adv"], clipped * s["adv"])
    away = s["ref"] - logp
    kl = torch.exp(away) - away - 1
    loss = torch.where(kept, s["weight"] * (c["kl"] * kl - gain), 0.0).sum(dtype=torch.float64).float().reshape(1)
    # d loss / d logp: the surrogate's branch that the minimum takes, and the KL term's
    slope = torch.where(ratio * s["adv"] <= clipped * s["adv"], -s["adv"] * ratio, 0.0)
    slope = s["weight"] * (slope + c["kl"] * (1 - torch.exp(away))) / tau
    dz = e * (-slope[:, None] / total)
    dz.scatter_add_(1, target, slope[:, None])
    dz = torch.where(kept[:, None], dz, 0.0)
    return {"logp": torch.where(kept, logp, 0.0), "loss": loss, "dlogits": dz.to(s["z"].dtype)}


def _dither(n, step):
    """A Weyl sequence over elements and steps, 20 bits: what the 8-bit states are rounded with."""
    i = torch.arange(n, dtype=torch.int64, device="cuda")
    return ((i * 0x9E3779B1 + step * 0x61C88647) & 0xFFFFFFFF) >> 12


def _to_e4m3(x, dither, least):
    """x rounded down to e4m3's grid after `dither` (20 bits of one grid step) was added."""
    a = x.abs()
    code = torch.where(a < 2.0 ** -6,
                       torch.floor(a * 512 + dither.float() * 2.0 ** -20) * 2.0 ** -9,
                       ((a.view(torch.int32).long() + dither) & ~0xFFFFF).to(torch.int32).view(torch.float32))
    if least:
        code = torch.where((a > 0) & (code == 0), 2.0 ** -9, code)
    return torch.copysign(code, x).to(torch.float8_e4m3fn)


def _blocks(x):
    n = x.numel()
    return torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)


def _quantise(x, codes, scales, dither, least):
    # the power of two that leaves a block's largest magnitude in [128, 256)
    top = _blocks(x.abs()).amax(1)
    scale = torch.where(top > 0, torch.ldexp(torch.ones_like(top), torch.frexp(top)[1] - 8), 0.0)
    y = (_blocks(x) / torch.where(top > 0, scale, 1.0)[:, None]).reshape(-1)[:x.numel()]
    codes.copy_(_to_e4m3(y, dither, least))
    scales.copy_(scale)


def _read(codes, scales):
    return codes.float() * scales.repeat_interleave(BLOCK)[:codes.numel()]


def _adamw_one(p, g, w, m, v, ms, vs, decay, step):
    h = HYPER
    c1, c2 = 1 - h["beta1"] ** step, 1 - h["beta2"] ** step
    g = g.float()
    m_old = m if ms is None else _read(m, ms)
    v_old = v if vs is None else _read(v, vs).square()
    m_new = h["beta1"] * m_old + (1 - h["beta1"]) * g
    v_new = h["beta2"] * v_old + (1 - h["beta2"]) * (g * g)
    root = torch.sqrt(v_new)
    x = p.float() if w is None else w
    x = x * (1 - h["lr"] * decay) - (m_new * (h["lr"] / c1)) / (root * (1 / math.sqrt(c2)) + h["eps"])
    p.copy_(x)
    if w is not None:
        w.copy_(x)
    if ms is None:
        m.copy_(m_new)
        v.copy_(v_new)
    else:
        dither = _dither(p.numel(), step)
        _quantise(m_new, m, ms, dither, False)
        _quantise(root, v, vs, dither ^ 0x80000, True)   # the root of v is what is held


def _adamw(s):
    if own:
        import token_routing_gb300 as moe
        if "opt" not in s:
            s["opt"] = moe.AdamW([dict(p=p, g=g, master=w, m=m, v=v, m_scale=ms, v_scale=vs, weight_decay=dec)
                                  for p, g, w, m, v, ms, vs, dec in zip(s["p"], s["g"], s["w"], s["m"], s["v"],
                                                                        s["ms"], s["vs"], s["decay"])],
                                 step=s["step"], rounding="weyl", **HYPER)
        s["opt"].step()
    else:
        s["step"] += 1
        [_adamw_one(*t, s["step"]) for t in zip(s["p"], s["g"], s["w"], s["m"], s["v"], s["ms"], s["vs"], s["decay"])]
    return {k: t for k, t in s["flat"].items() if k not in ("g16", "g32") and t.numel()}


# ------------------------------------------------------------------------------------ the least work

def _distinct(c):
    """Expected number of different tokens in a batch."""
    return float((1 - torch.pow(1 - _zipf(c["V"]), c["T"])).sum())


def work(case):
    c = case
    if c["op"] == "adamw":
        b = n = 0
        for k, p32, g32, _ in _tensors(c):
            per = 2 * (4 if p32 else 2) + (4 if g32 else 2)      # weight read and written, gradient read
            if c["master"] and not p32:
                per += 8 - 2                                     # the master instead of the weight is read
            per += 16 if c["bits"] == 32 else 4 + 16 / BLOCK
            b, n = b + k * per, n + k
        return {"bytes": b, "flops": 15 * n}
    T, V = c["T"], c["V"]
    if c["op"] == "embed":
        es = ES[c["dtype"]]
        return {"bytes": 4 * T + (_distinct(c) + T) * c["d"] * es, "flops": T * c["d"]}
    if c["op"] == "embed_grad":
        es, gs = ES[c["dtype"]], ES[c["grad"]]
        rows = 2 * _distinct(c) if c["accumulate"] else V
        return {"bytes": 4 * T + T * c["d"] * es + rows * c["d"] * gs, "flops": T * c["d"]}
    es = ES[c["dtype"]]
    if c["op"] == "logp":
        return {"bytes": T * V * es + 8 * T, "flops": 4 * T * V}
    kept = T * (1 - c["masked"])                                  # masked rows are written, not read
    return {"bytes": (kept + T) * V * es + 24 * T, "flops": 8 * kept * V}


# ------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s, c = prepare(case, seed), case
    return {"embed": _exact_embed, "embed_grad": _exact_embed_grad, "logp": _exact_logp, "policy": _exact_policy,
            "adamw": _exact_adamw}[c["op"]](s, c)


def _exact_embed(s, c):
    return torch.index_select(s["W"].double(), 0, s["ids"]) * c["scale"]


def _exact_embed_grad(s, c):
    # sorted tokens: the sum over each one's run is a difference of running sums' ends
    keep = s["ids"] != c["pad"]
    ids, order = torch.sort(s["ids"][keep].long())
    rows = s["dy"][keep][order].double() * c["scale"]
    values, counts = torch.unique_consecutive(ids, return_counts=True)
    out = s["dW"].double() if c["accumulate"] else torch.zeros(c["V"], c["d"], dtype=torch.float64, device="cuda")
    if values.numel():
        out[values] += torch.segment_reduce(rows, "sum", lengths=counts, axis=0)
    return out


def _exact_logp(s, c):
    return _logp_rows(s["z"], s["target"], c["temperature"])


def _exact_policy(s, c):
    """By the chain rule of the softmax on the loss's own derivative, which autograd gives for each token."""
    lp = _logp_rows(s["z"], s["target"], c["temperature"]).requires_grad_(True)
    kept = s["weight"] > 0
    lr, d = lp - s["old"].double(), s["ref"].double() - lp
    a = s["adv"].double()
    surrogate = torch.where(a >= 0, a * torch.exp(lr).clamp(max=1 + CLIP), a * torch.exp(lr).clamp(min=1 - CLIP))
    tokens = s["weight"].double() * (c["kl"] * (torch.expm1(d) - d) - surrogate)
    loss = tokens[kept].sum()
    (slope,) = torch.autograd.grad(loss, lp)
    dz = torch.empty(c["T"], c["V"], dtype=torch.float64, device="cuda")
    for a in range(0, c["T"], 512):
        z, t = s["z"][a:a + 512].double() / c["temperature"], s["target"][a:a + 512].long()
        p = torch.softmax(z, 1)
        hot = torch.nn.functional.one_hot(t, c["V"])
        dz[a:a + 512] = (slope[a:a + 512, None] / c["temperature"]) * (hot - p)
    return {"logp": torch.where(kept, lp.detach(), 0.0), "loss": loss.detach().reshape(1), "dlogits": dz}


def _grid64(x, dither, least):
    """|x| on e4m3's grid (three bits of a number's leading one, 2^-9 at the least), rounded down with the dither."""
    a = x.abs()
    unit = torch.pow(2.0, (torch.frexp(a)[1].double() - 4).clamp(min=-9))
    q = torch.floor(a / unit + dither.double() / 2 ** 20) * unit
    return torch.sign(x) * (torch.where(a > 0, q.clamp(min=2.0 ** -9), q) if least else q)


def _exact_adamw(s, c):
    h, step = HYPER, s["step"] + 1
    out = {k: t.double() for k, t in s["flat"].items() if k not in ("g16", "g32") and t.numel()}

    def put(key, view, x):
        at = view.storage_offset()
        out[key][at:at + x.numel()] = x

    def held(key, view, scales, x, dither, least):
        top = _blocks(x.abs()).amax(1)
        two = torch.where(top > 0, torch.exp2(torch.floor(torch.log2(top.clamp(min=1e-300))) - 7), 0.0)
        unit = torch.where(two > 0, two, 1.0).repeat_interleave(BLOCK)[:x.numel()]
        put(key, view, _grid64(x / unit, dither, least))
        put(key + "s", scales, two)

    for p, g, w, m, v, ms, vs, dec in zip(s["p"], s["g"], s["w"], s["m"], s["v"], s["ms"], s["vs"], s["decay"]):
        n, g = p.numel(), g.double()
        if ms is None:
            m1, v1 = m.double(), v.double()
        else:
            m1 = m.double() * ms.double().repeat_interleave(BLOCK)[:n]
            v1 = (v.double() * vs.double().repeat_interleave(BLOCK)[:n]) ** 2
        m1 = m1 + (1 - h["beta1"]) * (g - m1)
        v1 = v1 + (1 - h["beta2"]) * (g * g - v1)
        mean, square = m1 / (1 - h["beta1"] ** step), v1 / (1 - h["beta2"] ** step)
        x = (p if w is None else w).double()
        x = x - h["lr"] * (mean / (square.sqrt() + h["eps"]) + dec * x)
        put("p32" if p.dtype == torch.float32 else "p16", p, x)
        if w is not None:
            put("w", w, x)
        if ms is None:
            put("m", m, m1)
            put("v", v, v1)
        else:
            dither = _dither(n, step)
            held("m", m, ms, m1, dither, False)
            held("v", v, vs, v1.sqrt(), dither ^ 0x80000, True)
    return out
