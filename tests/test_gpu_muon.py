"""Orthogonalised updates (Muon) against the fp64 oracle.

The kernels round X, A and B to fp16 (one number, or two) at each step; the oracle takes the same
roundings at the same places in 64 bits, and its distance from the exact result is the size of error
that they make. A second set of roundings of that size is off by as much, so a kernel that rounds at
those places only stays within twice the distance in the Frobenius norm, and in one element within twice the
largest distance of any (elements are not alike: those along a strong direction are large in the first steps,
and so are their roundings, which stay with them; for 1 x 257 x 2048 the oracle's own largest is ten times its
root mean square). The output's own rounding is added.
"""
import numpy as np
import pytest
import torch

from oracle import operator_oracle as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
COEF = (3.4445, -4.7750, 2.0315)


def f64(t):
    return t.detach().double().cpu().numpy()


def make(count, rows, cols, dtype, seed=0, size=1e-3):
    g = torch.Generator().manual_seed(seed)
    r = min(3, rows, cols)
    u = torch.randn(count, rows, cols, generator=g) + torch.randn(count, rows, r, generator=g) @ torch.randn(count, r, cols, generator=g)
    return (u * size).to(DT[dtype])


def expected(u, precision, steps=5, coef=COEF):
    """(exact, size of the error in the Frobenius norm, and of the element that it is largest in) for one matrix."""
    ref = O.orth(u, steps, coef)
    off = O.orth(u, steps, coef, held=O.fp16_planes(1 if precision == "bf16" else 2)) - ref
    fro = np.sqrt((off * off).sum())
    # the scale's own rounding and that of the sums before it: 2^-20 of X, which a step leaves or shrinks,
    # but for small singular values, which grow with it
    own = 2.0 ** -20 * np.sqrt((ref * ref).sum())
    return ref, fro + own, np.abs(off).max() + 2.0 ** -20 * np.abs(ref).max()


def compare(got, u, precision, dtype, steps=5, coef=COEF, scale=1.0, base=None):
    """got = base - scale * orth(u), rounded to dtype."""
    for i in range(len(u)):
        ref, fro, one = expected(u[i], precision, steps, coef)
        want = ref if base is None else base[i] - scale * ref
        err = np.abs(got[i] - want)
        out = HALF[dtype] * np.abs(want) * 1.01 + (0 if base is None else 4 * 2.0 ** -24 * np.abs(base[i]))
        assert np.sqrt((np.maximum(err - out, 0) ** 2).sum()) <= 2 * scale * fro, (i, err.max(), fro)
        assert (err <= out + 2 * scale * one + 2.0 ** -40).all(), (i, err.max(), one)


def orthogonalize(moe, g, dtype, precision=None, steps=5, coef=COEF):
    n, r, c = g.shape
    cfg = moe.make_muon_config(n, r, c, dtype=dtype, grad_dtype="bf16" if g.dtype == torch.bfloat16 else "f32",
                               precision=precision, steps=steps, coef=coef)
    ws = torch.full((moe.muon_workspace_bytes(cfg),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN everywhere
    o = torch.full(g.shape, float("nan"), dtype=DT[dtype], device="cuda")
    moe.orthogonalize(cfg, g, o, ws)
    moe.get_error()
    return cfg, ws, o


SHAPES = [(1, 1, 1), (3, 1, 7), (2, 9, 1), (5, 45, 37), (2, 37, 45), (4, 64, 64), (1, 128, 200), (2, 130, 257),
          (2, 257, 130), (1, 300, 520), (3, 256, 256), (1, 16, 1000), (1, 1000, 24), (1, 520, 512), (2, 513, 300),
          (1, 257, 2048), (1, 2500, 130), (13, 600, 640), (7, 640, 520), (2, 35, 1500)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_orthogonalize(shape, dtype, grad, moe_lib, cuda_device):
    g = make(*shape, grad).cuda()
    cfg, ws, o = orthogonalize(moe_lib, g, dtype)
    compare(f64(o), f64(g), dtype, dtype)
    again = torch.empty_like(o)
    moe_lib.orthogonalize(cfg, g, again, ws)
    assert torch.equal(o, again)                          # bit for bit
    if dtype == grad:
        moe_lib.orthogonalize(cfg, g, g, ws)              # in place
        assert torch.equal(o, g)


@pytest.mark.parametrize("steps,coef", [(0, COEF), (1, COEF), (2, (1.5, -0.5, 0.0)), (8, (1.875, -1.25, 0.375))])
@pytest.mark.parametrize("precision", ["bf16", "f32"])
def test_steps_and_coefficients(steps, coef, precision, moe_lib, cuda_device):
    for shape in ((2, 70, 200), (2, 200, 70)):
        g = make(*shape, "f32").cuda()
        _, _, o = orthogonalize(moe_lib, g, "f32", precision, steps, coef)
        compare(f64(o), f64(g), precision, "f32", steps, coef)


def test_singular_values(moe_lib, cuda_device):
    """What it is for: singular values near one, the polar factor's directions."""
    g = make(2, 96, 160, "f32", seed=3).cuda()
    _, _, o = orthogonalize(moe_lib, g, "f32")
    s = torch.linalg.svdvals(o.double())
    assert float(s.min()) > 0.3 and float(s.max()) < 1.3


@pytest.mark.parametrize("size", [1e-12, 1e-5, 1.0, 1e6, 1e15])
def test_sizes_of_gradients(size, moe_lib, cuda_device):
    g = make(2, 60, 80, "f32", size=size).cuda()
    for precision in ("bf16", "f32"):
        _, _, o = orthogonalize(moe_lib, g, "f32", precision)
        compare(f64(o), f64(g), precision, "f32")


@pytest.mark.parametrize("shape", [(6, 40, 64), (6, 300, 37)])
@pytest.mark.parametrize("precision", ["bf16", "f32"])
def test_matrices_stand_apart(shape, precision, moe_lib, cuda_device):
    """Zeros stay zeros; a matrix with NaN, an infinity or elements whose squares pass fp32 is NaN; the
    others are what they are alone."""
    g = make(*shape, "f32").cuda()
    g[1] = 0
    g[2, 5, 7], g[3, shape[1] - 1, shape[2] - 1], g[4, 0, 0] = float("nan"), float("inf"), 1e30
    _, _, o = orthogonalize(moe_lib, g, "f32", precision)
    assert (o[1] == 0).all()
    assert torch.isnan(o[2:5]).all()
    for i in (0, 5):
        _, _, alone = orthogonalize(moe_lib, g[i:i + 1].contiguous(), "f32", precision)
        assert torch.equal(alone[0], o[i])


def test_one_strong_direction(moe_lib, cuda_device):
    """Singular values from 1 to 1e-4 of the largest: the small ones are lifted, with their rounding."""
    g = torch.Generator().manual_seed(4)
    left, right = (torch.linalg.qr(torch.randn(64, 64, generator=g, dtype=torch.float64))[0] for _ in range(2))
    u = ((left * torch.logspace(0, -4, 64, dtype=torch.float64)) @ right).float()[None].cuda()
    for precision in ("bf16", "f32"):
        _, _, o = orthogonalize(moe_lib, u, "f32", precision)
        compare(f64(o), f64(u), precision, "f32")


def steps_of(moe, shape, dtype, grad, master, nesterov, precision=None, n=3, **dev):
    count, rows, cols = shape
    p = make(*shape, dtype, seed=7, size=0.02).cuda()
    t = dict(p=p.clone(), g=make(*shape, grad, seed=8).cuda(), weight_decay=0.1)
    if master:
        t["master"] = p.float() + 1e-4 * torch.randn(p.shape, generator=torch.Generator().manual_seed(9)).cuda()
    x = f64(t["master"] if master else t["p"])
    m = np.zeros(shape)
    opt = moe.Muon([t], lr=0.02, momentum=0.9, nesterov=nesterov, precision=precision)
    t = opt.tensors[0]
    prec = precision or dtype
    scale = 0.2 * np.sqrt(max(rows, cols))
    for k in range(n):
        t["g"].copy_(make(*shape, grad, seed=20 + k).cuda())
        lr, gs = 0.02, 1.0
        if dev:
            lr, gs = 0.01 * (k + 1), 0.5 + k
            opt.step(lr=torch.tensor([lr], device="cuda"), grad_scale=torch.tensor([gs], device="cuda"))
            lr, gs = float(np.float32(lr)), float(np.float32(gs))
        else:
            opt.step()
            lr = float(np.float32(lr))
        g, mu = f64(t["g"]) * gs, float(np.float32(0.9))
        m = mu * m + g
        got_m = f64(t["m"])
        assert (np.abs(got_m - m) <= 4 * 2.0 ** -24 * (np.abs(m) + np.abs(g)) * (k + 1)).all()
        m = got_m
        u = g + mu * m if nesterov else m
        base = x * (1 - lr * float(np.float32(0.1)))
        move = lr * float(np.float32(scale))
        now = t["master"] if master else t["p"]
        compare(f64(now), u, prec, "f32" if master else dtype, scale=move, base=base)
        if master:
            assert torch.equal(t["p"], t["master"].to(t["p"].dtype))
        x = f64(now)
    moe.get_error()


@pytest.mark.parametrize("shape", [(2, 45, 37), (1, 24, 200), (3, 264, 96)])
@pytest.mark.parametrize("dtype,grad,master", [("bf16", "bf16", False), ("bf16", "bf16", True), ("f32", "f32", False),
                                               ("bf16", "f32", True), ("f32", "bf16", True)])
def test_step(shape, dtype, grad, master, moe_lib, cuda_device):
    steps_of(moe_lib, shape, dtype, grad, master, True)
    steps_of(moe_lib, shape, dtype, grad, master, False, n=1)


def test_step_with_device_scalars(moe_lib, cuda_device):
    steps_of(moe_lib, (2, 45, 40), "bf16", "bf16", True, True, dev=True)
    steps_of(moe_lib, (2, 45, 40), "f32", "f32", False, False, precision="bf16", dev=True)


def test_matrix_and_stack(moe_lib, cuda_device):
    """[rows, cols] is a stack of one; several tensors in one optimiser share its workspace."""
    moe = moe_lib
    ps = [make(1, 48, 64, "f32", seed=i, size=0.02)[0].cuda() for i in range(2)] + [make(3, 20, 90, "f32", size=0.02).cuda()]
    gs = [make(*(p.shape if p.dim() == 3 else (1, *p.shape)), "f32", seed=5).reshape(p.shape).cuda() for p in ps]
    both = [p.clone() for p in ps]
    moe.Muon([dict(p=p, g=g) for p, g in zip(both, gs)]).step()
    for p, g, b in zip(ps, gs, both):
        moe.Muon([dict(p=p, g=g)]).step()
        assert torch.equal(p, b)
    moe.get_error()


@pytest.mark.parametrize("shape", [(2, 256, 320), (3, 100, 700), (3, 40, 33)])
def test_graph_and_two_streams(shape, moe_lib, cuda_device):
    """A captured step, replayed while another optimiser steps on its own stream."""
    moe = moe_lib
    made = [[make(*shape, "bf16", seed=i, size=0.02).cuda(), make(*shape, "bf16", seed=10 + i).cuda()] for i in range(2)]
    want = []
    for p, g in made:
        q = p.clone()
        opt = moe.Muon([dict(p=q, g=g)])
        for _ in range(4):
            opt.step()
        want.append((q, opt.tensors[0]["m"]))
    torch.cuda.synchronize()
    (p0, g0), (p1, g1) = made
    a, b = moe.Muon([dict(p=p0, g=g0)]), moe.Muon([dict(p=p1, g=g1)])
    s0, s1 = torch.cuda.Stream(), torch.cuda.Stream()
    s0.wait_stream(torch.cuda.current_stream())
    s1.wait_stream(torch.cuda.current_stream())
    a.step(stream=s0)                                      # eager first
    s0.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s0):
        a.step()
    for _ in range(3):
        with torch.cuda.stream(s0):
            graph.replay()
        b.step(stream=s1)
    b.step(stream=s1)
    torch.cuda.synchronize()
    for opt, (p, m) in zip((a, b), want):
        assert torch.equal(opt.tensors[0]["p"], p) and torch.equal(opt.tensors[0]["m"], m)
    moe.get_error()


@pytest.mark.parametrize("shape", [(1, 300, 704), (3, 704, 336), (30, 520, 304), (40, 300, 600), (40, 600, 304)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tiles_of_every_width(shape, dtype, moe_lib, cuda_device):
    """Few matrices, whose tiles are narrow, and many, whose tiles are wide; four of them are looked at."""
    g = make(*shape, dtype).cuda()
    _, _, o = orthogonalize(moe_lib, g, dtype)
    pick = sorted({0, shape[0] // 2, max(0, shape[0] - 2), shape[0] - 1})
    compare(f64(o)[pick], f64(g)[pick], dtype, dtype)
    assert torch.isfinite(o.float()).all()
