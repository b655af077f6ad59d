"""8-bit AdamW states under both rounding rules, and runs of many units of one tensor, against the
fp64 oracle, element by element.

Tolerances count roundings of 2^-24 (U): m and v are two products with rounded constants (4 on each
term) and a sum; the update is a product, a square root, an fma and an approximate division (2
units), with three rounded constants: 24 of its own size; x takes 3 more. p is x rounded once to its
type. A held value is the oracle's for a value within 2^-20 of its own and a dither one count to
either side (the kernel's share of the way is cut off to 20 bits); a block's scale is the oracle's
for a largest magnitude within 2^-20."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 2 ** 20                    # elements that the oracle takes at a time


def f64(t):
    return t.detach().double().cpu().numpy()


def tensors(kinds, g, decay=0.1):
    """kinds: (elements, weight type, gradient type, master)."""
    out = []
    for i, (n, dtype, grad, master) in enumerate(kinds):
        size = torch.exp(torch.randn(n, generator=g, device="cuda") * 2) * 1e-3
        t = dict(p=torch.randn(n, generator=g, device="cuda").to(DT[dtype]),
                 g=(torch.randn(n, generator=g, device="cuda") * size).to(DT[grad]), weight_decay=decay * (i % 2))
        if master:
            t["master"] = torch.randn(n, generator=g, device="cuda")
        out.append(t)
    return out


def part(t, k, a, b):
    return f64(t[k][a:b].float())


def moments(t, a, b):
    m, v = part(t, "m", a, b), part(t, "v", a, b)
    if t["m_scale"] is None:
        return m, v
    ms, vs = (np.repeat(f64(t[k][a // O.BLOCK:-(-b // O.BLOCK)]), O.BLOCK)[:b - a] for k in ("m_scale", "v_scale"))
    return m * ms, (v * vs) ** 2


def check_held(codes, scale, y, e, d, root, even):
    lo, hi = O.block_scale(y * (1 - 2.0 ** -20)), O.block_scale(y * (1 + 2.0 ** -20))
    assert ((scale == lo) | (scale == hi)).all()
    top = np.repeat(scale, O.BLOCK)[:len(y)]
    some = top > 0
    u, e = np.where(some, y / np.where(some, top, 1), 0), np.where(some, e / np.where(some, top, 1), 0)
    e = e + np.abs(u) * 2.0 ** -20 + 2.0 ** -30
    low = O.held(np.maximum(np.abs(u) - e, 0), np.maximum(d - 1, 0), root, even)
    high = O.held(np.abs(u) + e, d + 1, root, even)
    sure = np.abs(u) > e
    assert (np.abs(codes) >= np.where(sure, low, 0)).all() and (np.abs(codes) <= high).all()
    assert (np.sign(codes)[sure & (codes != 0)] == np.sign(u)[sure & (codes != 0)]).all()


def check_step(opt, rounding="even", every=1):
    """One step, checked on every so many chunks of a tensor and on its last."""
    cfg = opt.cfg
    b1, b2, eps, lr = cfg.beta1, cfg.beta2, np.float64(np.float32(cfg.eps)), cfg.lr
    before = [{k: None if t[k] is None else t[k].clone() for k in ("p", "master", "m", "v", "m_scale", "v_scale")}
              for t in opt.tensors]
    step = opt.steps_done() + 1
    opt.step()
    assert opt.steps_done() == step
    for t, old in zip(opt.tensors, before):
        n, key = t["p"].numel(), "p" if t["master"] is None else "master"
        if t["master"] is not None:
            assert torch.equal(t["p"], t["master"].to(t["p"].dtype))
        for a in range(0, n, CHUNK):
            b = min(n, a + CHUNK)
            if a // CHUNK % every and b < n:
                continue
            x, grad, (m, v) = part(old, key, a, b), part(t, "g", a, b), moments(old, a, b)
            nx, nm, nv, up = O.adamw(x, grad, m, v, step, lr, b1, b2, eps, np.float64(np.float32(t["weight_decay"])))
            tm = (6 * U) * (b1 * np.abs(m) + (1 - b1) * np.abs(grad))
            tv = (8 * U) * nv + 1e-44
            with np.errstate(divide="ignore", invalid="ignore"):
                tx = up * 24 * U + np.where(nm != 0, up * tm / np.abs(nm), 0) + 3 * U * np.abs(x) + U * np.abs(nx)
            if key == "p" and t["p"].dtype == torch.bfloat16:
                tx = tx + np.abs(nx) * 2.0 ** -8 * 1.01
            assert (np.abs(part(t, key, a, b) - nx) <= tx + 1e-44).all()
            if t["m_scale"] is None:
                assert (np.abs(part(t, "m", a, b) - nm) <= tm + 1e-44).all()
                assert (np.abs(part(t, "v", a, b) - nv) <= tv).all()
                continue
            dm, dv = (O.dither if rounding == "even" else O.weyl)(b - a, step, a)
            blocks = slice(a // O.BLOCK, -(-b // O.BLOCK))
            check_held(part(t, "m", a, b), f64(t["m_scale"][blocks]), nm, tm, dm, False, rounding == "even")
            check_held(part(t, "v", a, b), f64(t["v_scale"][blocks]), np.sqrt(nv), np.sqrt(nv) * 8 * U, dv, True,
                       rounding == "even")


SHORT = [(1, "f32", "f32", False), (255, "bf16", "bf16", False), (256, "bf16", "f32", True), (257, "f32", "bf16", False),
         (2048, "bf16", "bf16", True), (5001, "bf16", "f32", False), (0, "f32", "f32", False), (77, "f32", "f32", True)]


@pytest.mark.parametrize("rounding", ["even", "weyl"])
def test_rounding_rules(rounding, moe_lib, cuda_device):
    """Fresh states, in every kind of tensor, over steps with gradients of their own."""
    g = torch.Generator(device="cuda").manual_seed(0)
    opt = moe_lib.AdamW(tensors(SHORT, g), lr=1e-2, beta2=0.95, bits=8, rounding=rounding)
    for _ in range(4):
        check_step(opt, rounding)
        for t in opt.tensors:
            t["g"].mul_(torch.randn(t["g"].numel(), generator=g, device="cuda").to(t["g"].dtype))


def test_rounding_of_resumed_states(moe_lib, cuda_device):
    """8-bit states handed over with their step count; the default rule is the even one."""
    g = torch.Generator(device="cuda").manual_seed(1)
    for kw in (dict(), dict(rounding="even"), dict(rounding="weyl")):
        first = moe_lib.AdamW(tensors(SHORT, g), bits=8, **kw)
        first.step()
        states = [{k: t[k] for k in ("p", "g", "master", "m", "v", "m_scale", "v_scale")} for t in first.tensors]
        opt = moe_lib.AdamW(states, beta1=0.8, step=20, **kw)
        check_step(opt, kw.get("rounding", "even"))


def test_rounding_leaves_wide_states_alone(moe_lib, cuda_device):
    a, b = (moe_lib.AdamW(tensors(SHORT, torch.Generator(device="cuda").manual_seed(2)), rounding=r)
            for r in ("even", "weyl"))
    a.step()
    b.step()
    for x, y in zip(a.tensors, b.tensors):
        assert torch.equal(x["p"], y["p"]) and torch.equal(x["m"], y["m"]) and torch.equal(x["v"], y["v"])


def test_weyl_rounding_of_values_that_are_not_finite(moe_lib, cuda_device):
    """Held as NaN, the rest of the block as it would be."""
    a, b = (tensors([(1000, "f32", "f32", False)], torch.Generator(device="cuda").manual_seed(5)) for _ in "ab")
    bad = [3, 400, 401, 999]
    for t in (a, b):
        t[0]["g"][bad] = 0.0
    b[0]["g"][torch.tensor(bad)] = torch.tensor([float("inf"), float("nan"), -float("inf"), float("nan")]).cuda()
    oa, ob = (moe_lib.AdamW(t, bits=8, rounding="weyl") for t in (a, b))
    for _ in range(2):
        oa.step()
        ob.step()
    rest = [i for i in range(1000) if i not in bad]
    for k in ("p", "m", "v"):
        x, y = oa.tensors[0][k].float(), ob.tensors[0][k].float()
        assert torch.equal(x[rest], y[rest]) and not torch.isfinite(y[bad]).any()


KINDS = [(p, g, master) for p in ("f32", "bf16") for g in ("f32", "bf16") for master in (False, True)]


@pytest.mark.parametrize("bits,rounding", [(32, "even"), (8, "even"), (8, "weyl")])
@pytest.mark.parametrize("n", [170_001, 410_777, 1_000_003])
def test_runs_of_many_units(n, bits, rounding, moe_lib, cuda_device):
    """Every kind of tensor in runs of several units a warp: the next unit's loads pass under this one's
    arithmetic, the scales go out together, and the tensor's end cuts a run and a unit short."""
    g = torch.Generator(device="cuda").manual_seed(n)
    opt = moe_lib.AdamW(tensors([(n + 259 * i, *kind) for i, kind in enumerate(KINDS)], g), lr=1e-2, bits=bits,
                        rounding=rounding)
    for _ in range(2):
        check_step(opt, rounding)
        for t in opt.tensors:
            t["g"].mul_(torch.randn(t["g"].numel(), generator=g, device="cuda").to(t["g"].dtype))


@pytest.mark.parametrize("bits,rounding,n", [(32, "even", 24_300_001), (8, "even", 55_000_001), (8, "weyl", 55_000_001)])
def test_longest_runs(bits, rounding, n, moe_lib, cuda_device):
    """The longest runs (16 eights of units, 32 with 8-bit states), over a thousand of them in one launch: the
    step is then counted by a launch of its own, once a call."""
    g = torch.Generator(device="cuda").manual_seed(bits)
    opt = moe_lib.AdamW(tensors([(n, "bf16", "bf16", True), (n * 3 // 5, "bf16", "f32", False)], g), lr=1e-2,
                        bits=bits, rounding=rounding)
    for _ in range(2):
        check_step(opt, rounding, every=7)


def test_long_runs_beside_short_ones(moe_lib, cuda_device):
    """Both widths of states in one call, tensors from one element to millions."""
    g = torch.Generator(device="cuda").manual_seed(11)
    kinds = [(3_000_001, "bf16", "bf16", True), (1, "f32", "f32", False), (2_000_037, "f32", "bf16", False),
             (65_536 * 8, "bf16", "f32", True), (300, "bf16", "bf16", False), (16_384 * 2, "f32", "f32", False)]
    ts = tensors(kinds + kinds, g)
    for t in ts[:len(kinds)]:
        codes, scales = torch.zeros(t["p"].numel(), device="cuda"), torch.zeros(-(-t["p"].numel() // O.BLOCK), device="cuda")
        t.update(m=codes.to(torch.float8_e4m3fn), v=codes.to(torch.float8_e4m3fn), m_scale=scales, v_scale=scales.clone())
    opt = moe_lib.AdamW(ts, lr=3e-3)
    for _ in range(2):
        check_step(opt)
