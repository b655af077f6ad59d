"""AdamW over many tensors against the fp64 oracle.

Tolerances count roundings of 2^-24: m and v are two products with rounded constants (4 on each
term) and a sum; the update is a product, a square root, an fma and an approximate division
(2 units), with three rounded constants: 24 of its own size; x takes 3 more. p is x rounded once
to its type. 8-bit states: the held value is that of the oracle's rule for a value within 2^-20
of its own (the fp32 roundings before it)."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def gradient(n, dtype, g):
    x = torch.randn(n, generator=g) * 1e-3
    return (x * torch.exp(torch.randn(n, generator=g) * 2)).to(DT[dtype]).cuda()


def tensors(sizes, dtype, grad, master, g, decay=0.1):
    out = []
    for i, n in enumerate(sizes):
        p = torch.randn(n, generator=g).to(DT[dtype]).cuda()
        t = dict(p=p, g=gradient(n, grad, g), weight_decay=decay if i % 2 == 0 else 0.0)
        if master:
            t["master"] = torch.randn(n, generator=g).cuda()
        out.append(t)
    return out


def states(t):
    """(m, v) as fp64, from either form."""
    if t["m_scale"] is None:
        return f64(t["m"]), f64(t["v"])
    n = t["p"].numel()
    ms, vs = (np.repeat(f64(t[k]), O.BLOCK)[:n] for k in ("m_scale", "v_scale"))
    return f64(t["m"].float()) * ms, (f64(t["v"].float()) * vs) ** 2


def check_step(moe, opt):
    cfg = opt.cfg
    b1, b2, eps, lr = cfg.beta1, cfg.beta2, np.float64(np.float32(cfg.eps)), cfg.lr
    before = []
    for t in opt.tensors:
        x = t["master"] if t["master"] is not None else t["p"]
        before.append((f64(x), f64(t["g"]), *states(t)))
    step = opt.steps_done() + 1
    opt.step()
    assert opt.steps_done() == step
    for t, (x, g, m, v) in zip(opt.tensors, before):
        nx, nm, nv, up = O.adamw(x, g, m, v, step, lr, b1, b2, eps, np.float64(np.float32(t["weight_decay"])))
        tm = (6 * U) * (b1 * np.abs(m) + (1 - b1) * np.abs(g))
        tv = (8 * U) * nv + 1e-44
        # an error of m passes to the update in proportion, one of v by half
        with np.errstate(divide="ignore", invalid="ignore"):
            tx = up * 24 * U + np.where(nm != 0, up * tm / np.abs(nm), 0) + 3 * U * np.abs(x) + U * np.abs(nx)
        got = f64(t["master"] if t["master"] is not None else t["p"])
        if t["master"] is None and t["p"].dtype == torch.bfloat16:
            tx = tx + np.abs(nx) * 2.0 ** -8 * 1.01
        assert (np.abs(got - nx) <= tx + 1e-44).all(), (np.abs(got - nx) - tx).max()
        if t["master"] is not None:
            assert torch.equal(t["p"], t["master"].to(t["p"].dtype))
        if t["m_scale"] is None:
            assert (np.abs(f64(t["m"]) - nm) <= tm + 1e-44).all() and (np.abs(f64(t["v"]) - nv) <= tv).all()
            continue
        n = len(x)
        for codes, scale, y, d, root, e in ((t["m"], t["m_scale"], nm, O.dither(n, step)[0], False, tm),
                                            (t["v"], t["v_scale"], np.sqrt(nv), O.dither(n, step)[1], True,
                                             np.sqrt(nv) * 8 * U)):
            sc = O.block_scale(y)
            assert (np.abs(f64(scale) - sc) <= sc * 2.0 ** -20).all()
            top = np.repeat(sc, O.BLOCK)[:n]
            some = top > 0
            got = f64(codes.float())
            u, e = np.where(some, y / np.where(some, top, 1), 0), np.where(some, e / np.where(some, top, 1), 0)
            e = e + np.abs(u) * 2.0 ** -20 + 2.0 ** -30
            # |held| grows with |y| and with the dither: bounds at either end of the tolerance
            a, b = O.held(np.maximum(np.abs(u) - e, 0), np.maximum(d - 1, 0), root), O.held(np.abs(u) + e, d + 1, root)
            assert (np.abs(got) >= np.where(np.abs(u) > e, a, 0)).all() and (np.abs(got) <= b).all()
            sure = np.abs(u) > e
            assert (np.sign(got)[sure & (got != 0)] == np.sign(u)[sure & (got != 0)]).all()


SIZES = [1, 7, 8, 9, 255, 256, 257, 1000, 2048, 5000, 37 * 45]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,grad,master", [("f32", "f32", False), ("bf16", "bf16", False), ("bf16", "f32", True),
                                               ("bf16", "bf16", True), ("f32", "bf16", False)])
def test_steps(bits, dtype, grad, master, moe_lib, cuda_device):
    g = torch.Generator().manual_seed(0)
    opt = moe_lib.AdamW(tensors(SIZES, dtype, grad, master, g), lr=1e-2, bits=bits)
    for _ in range(4):
        check_step(moe_lib, opt)
        for t in opt.tensors:
            t["g"].copy_(gradient(t["g"].numel(), grad, g))
    moe_lib.get_error()


def test_mixed_tensors_in_one_call(moe_lib, cuda_device):
    """Types, masters, state widths and decays side by side, in more tensors than one launch takes."""
    g = torch.Generator().manual_seed(1)
    ts = []
    for i in range(700):
        n = [0, 1, 33, 300, 513][i % 5]
        dtype, grad = ("bf16", "f32")[i % 2], ("bf16", "f32")[(i // 2) % 2]
        (t,) = tensors([n], dtype, grad, dtype == "bf16" and i % 3 == 0, g, decay=0.01 * (i % 4))
        if i % 7 < 3:
            blocks = -(-n // O.BLOCK)
            t.update(m=torch.zeros(n, device="cuda").to(torch.float8_e4m3fn),
                     v=torch.zeros(n, device="cuda").to(torch.float8_e4m3fn),
                     m_scale=torch.zeros(blocks, device="cuda"), v_scale=torch.zeros(blocks, device="cuda"))
        ts.append(t)
    opt = moe_lib.AdamW(ts, lr=3e-3, weight_decay=0.1)
    for _ in range(2):
        check_step(moe_lib, opt)


def test_resumed_states(moe_lib, cuda_device):
    """States and a step count from elsewhere: the bias corrections of step 1001."""
    g = torch.Generator().manual_seed(2)
    ts = tensors([900], "f32", "f32", False, g)
    ts[0].update(m=torch.randn(900, generator=g).cuda() * 1e-3, v=torch.rand(900, generator=g).cuda() * 1e-6)
    opt = moe_lib.AdamW(ts, lr=1e-2, beta2=0.999, step=1000)
    for _ in range(3):
        check_step(moe_lib, opt)


@pytest.mark.parametrize("beta1,beta2", [(0.0, 0.0), (0.0, 0.99), (0.9, 0.9999)])
def test_betas(beta1, beta2, moe_lib, cuda_device):
    g = torch.Generator().manual_seed(3)
    opt = moe_lib.AdamW(tensors([600], "f32", "f32", False, g), beta1=beta1, beta2=beta2, eps=1e-6)
    for _ in range(3):
        check_step(moe_lib, opt)


def test_learning_rate_and_gradient_scale_on_the_device(moe_lib, cuda_device):
    g = torch.Generator().manual_seed(4)
    opt = moe_lib.AdamW(tensors([700, 40], "f32", "f32", False, g), lr=1.0)
    lr, gs = torch.tensor([5e-3], device="cuda"), torch.tensor([0.25], device="cuda")
    before = [f64(t["p"]) for t in opt.tensors]
    ref = [O.adamw(x, f64(t["g"]) * 0.25, 0.0, 0.0, 1, float(lr), 0.9, 0.999, 1e-8, np.float64(np.float32(t["weight_decay"])))
           for x, t in zip(before, opt.tensors)]
    opt.step(lr=lr, grad_scale=gs)
    for t, (nx, nm, nv, up), x in zip(opt.tensors, ref, before):
        assert (np.abs(f64(t["p"]) - nx) <= up * 32 * U + 4 * U * np.abs(x) + 1e-44).all()
        assert (np.abs(f64(t["m"]) - nm) <= 6 * U * np.abs(nm) + 1e-44).all()


def test_no_tensors_counts_the_step(moe_lib, cuda_device):
    opt = moe_lib.AdamW([])
    opt.step()
    opt.step()
    assert opt.steps_done() == 2
    opt = moe_lib.AdamW([dict(p=torch.zeros(0, device="cuda"), g=torch.zeros(0, device="cuda"))], bits=8)
    opt.step()
    assert opt.steps_done() == 1


def test_values_that_are_not_finite(moe_lib, cuda_device):
    """An infinite or NaN gradient makes its own weight NaN and, with 8-bit states, leaves the other
    255 elements of its block as they would be."""
    for bits in (32, 8):
        a, b = (tensors([1000], "f32", "f32", False, torch.Generator().manual_seed(5)) for _ in "ab")
        bad = [3, 400, 401, 999]
        for t in (a, b):
            t[0]["g"][bad] = 0.0
        b[0]["g"][torch.tensor(bad)] = torch.tensor([float("inf"), float("nan"), -float("inf"), float("nan")]).cuda()
        oa, ob = moe_lib.AdamW(a, bits=bits), moe_lib.AdamW(b, bits=bits)
        for _ in range(2):
            oa.step()
            ob.step()
        rest = [i for i in range(1000) if i not in bad]
        for k in ("p", "m", "v"):
            x, y = oa.tensors[0][k].float(), ob.tensors[0][k].float()
            assert torch.equal(x[rest], y[rest]) and not torch.isfinite(y[bad]).any()


def test_zero_gradients_and_blocks(moe_lib, cuda_device):
    """All-zero blocks keep scale and codes zero; a gradient far below its block's largest still
    moves its weight by no more than lr a step (sqrt(v) never becomes 0)."""
    g = torch.Generator().manual_seed(6)
    ts = tensors([1024], "f32", "f32", False, g, decay=0.0)
    ts[0]["g"].zero_()
    ts[0]["g"][512:768] = 1e-9
    ts[0]["g"][512] = 1.0
    opt = moe_lib.AdamW(ts, lr=1e-2, bits=8)
    p0 = ts[0]["p"].clone()
    for i in range(50):
        opt.step()
    t = opt.tensors[0]
    assert torch.equal(t["p"][:512], p0[:512]) and torch.equal(t["p"][768:], p0[768:])
    assert t["m_scale"].tolist()[:2] == [0, 0] and (t["v"].float()[:512] == 0).all()
    assert (t["v"].float()[512:768] > 0).all()
    moved = (t["p"] - p0)[512:768].abs()
    assert moved.max() <= 50 * 1e-2 * 1.2 and float(moved[0]) > 0.3


def test_8bit_second_moment_follows_the_gradient(moe_lib, cuda_device):
    """beta2 = 0.999 moves sqrt(v) by under 0.1 % a step, far below half a step of e4m3 (3 to 6 %):
    rounding to nearest would leave it where it began. With the dither it follows: gradients whose
    size doubles for half of each block must show in v, on average to 2 %, after 3000 steps."""
    n = 4096
    g = torch.Generator().manual_seed(7)
    size = torch.exp(torch.randn(n, generator=g)).cuda() * 1e-3
    p = torch.zeros(n, device="cuda")
    t = dict(p=p, g=size.clone())
    opt = moe_lib.AdamW([t], lr=0.0, bits=8)
    ref = np.zeros(n)
    for phase in (1.0, 2.0):
        up = torch.where(torch.arange(n, device="cuda") % 2 == 0, phase, 1.0)
        t["g"].copy_(size * up)
        gg = f64(t["g"]) ** 2
        for _ in range(3000):
            opt.step()
        ref = gg + (ref - gg) * 0.999 ** 3000
        _, v = states(opt.tensors[0])
        assert abs((v / ref).mean() - 1) < 0.02


def test_repeats_bit_for_bit(moe_lib, cuda_device):
    runs = []
    for _ in range(2):
        g = torch.Generator().manual_seed(8)
        opt = moe_lib.AdamW(tensors([5000, 77, 20000], "bf16", "bf16", True, g), bits=8)
        for _ in range(3):
            opt.step()
        runs.append(opt.tensors)
    for a, b in zip(*runs):
        for k in ("p", "master", "m_scale", "v_scale"):
            assert torch.equal(a[k], b[k])
        assert torch.equal(a["m"].view(torch.uint8), b["m"].view(torch.uint8))
        assert torch.equal(a["v"].view(torch.uint8), b["v"].view(torch.uint8))


def test_tensors_past_two_billion_elements(moe_lib, cuda_device):
    n = 2 ** 31 + 2 ** 20 + 5
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 2 ** 31 - 1, 2 ** 31, n - 1], device="cuda")
    g[at] = torch.tensor([1.0, -2.0, 3.0, -4.0], device="cuda").bfloat16()
    opt = moe_lib.AdamW([dict(p=p, g=g)], lr=0.5, bits=8)
    opt.step()
    # the first step is lr against the gradient's sign
    assert p[at].float().tolist() == [-0.5, 0.5, -0.5, 0.5]
    assert int(torch.count_nonzero(p[:2 ** 30])) == 1 and int(torch.count_nonzero(p[2 ** 30:2 ** 31])) == 1
    assert int(torch.count_nonzero(p[2 ** 31:])) == 2


def test_graph_counts_its_steps(moe_lib, cuda_device):
    """Captured once and replayed: the step count, the bias corrections and the dither advance on the
    device, and the learning rate is read there."""
    a, b = (tensors([3000, 70], "bf16", "f32", True, torch.Generator().manual_seed(9)) for _ in "ab")
    lr = torch.tensor([1e-2], device="cuda")
    oa, ob = moe_lib.AdamW(a, bits=8), moe_lib.AdamW(b, bits=8)
    oa.step(lr=lr)
    ob.step(lr=lr)
    torch.cuda.synchronize()
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        ob.step(lr=lr, stream=st)
    assert ob.steps_done() == 1
    for i in range(4):
        lr.fill_(1e-2 / (i + 1))
        oa.step(lr=lr)
        graph.replay()
    torch.cuda.synchronize()
    assert oa.steps_done() == ob.steps_done() == 5
    for x, y in zip(oa.tensors, ob.tensors):
        for k in ("p", "master", "m_scale", "v_scale"):
            assert torch.equal(x[k], y[k])
        assert torch.equal(x["v"].view(torch.uint8), y["v"].view(torch.uint8))
