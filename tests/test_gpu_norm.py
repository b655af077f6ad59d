"""Layer norm and its gradient against the fp64 oracle.

Tolerances count roundings (u = 2^-24 in fp32, HALF for one rounding to the output type). A sum over a
row is added up in at most 80 additions one after another (32 to a thread, or d / 1024, then 5, then 32),
so it is off by 80 u of the sum of magnitudes."""
import numpy as np
import pytest
import torch

from oracle import operator_oracle as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 2.0 ** -24
N = 80 * U


def f64(t):
    return t.detach().double().cpu().numpy()


def make(T, d, dtype, params, seed=0, offset=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, d, generator=g) + offset * torch.randn(T, 1, generator=g)).to(DT[dtype])
    r = torch.randn(T, d, generator=g).to(DT[dtype])
    gain, bias = (torch.randn(d, generator=g).to(DT[params]) for _ in range(2))
    dy, dt = (torch.randn(T, d, generator=g).to(DT[dtype]) for _ in range(2))
    return [t.cuda() for t in (x, r, gain, bias, dy, dt)]


def close(got, ref, tol):
    err = np.abs(got - ref)
    assert (err <= tol).all(), (err.max(), (err / tol).max())


def check_forward(moe, T, d, dtype, params, residual, eps=1e-5, plain=False, offset=1.0):
    x, r, gain, bias, _, _ = make(T, d, dtype, params, offset=offset)
    c = moe.make_norm_config(T, d, eps=eps, dtype=dtype, param_dtype=params)
    y = torch.full_like(x, float("nan"))
    total = torch.full_like(x, float("nan")) if residual else None
    mean, rstd = torch.full((T,), float("nan"), device="cuda"), torch.full((T,), float("nan"), device="cuda")
    moe.layer_norm(c, x, None if plain else gain, None if plain else bias, y, residual=r if residual else None,
                   total=total, mean=mean, rstd=rstd)
    moe.get_error()
    s = f64(x) + f64(r) if residual else f64(x)
    gn, bn = (np.ones(d), np.zeros(d)) if plain else (f64(gain), f64(bias))
    ref, rm, rr = O.norm(s, gn, bn, float(np.float32(eps)))
    dm = N * np.abs(s).mean(axis=1) + 2 * U * np.abs(rm)
    var = 1 / (rr * rr)                                   # eps and all: the smallest it can be off
    rv = N + 8 * U + dm * dm / var
    # x + residual is rounded to fp32: element i by U |s_i|, and with it the mean by up to U mean|s|, so s_i - mean by
    # own_i = U (|s_i| + mean|s|). The mean of the squares of e_i = s_i - mean changes by mean(2 e_i own_i + own_i^2), at
    # most 2 sqrt(mean e^2) sqrt(mean own^2) + mean own^2 (Cauchy), relative to var >= mean e^2 by 2 q + q^2 with
    # q = sqrt(mean own^2 / var).
    own = U * (np.abs(s) + np.abs(s).mean(axis=1, keepdims=True)) if residual else np.zeros_like(s)
    q = np.sqrt((own * own).mean(axis=1) / var)
    rv = rv + 2 * q + q * q
    close(f64(mean), rm, dm)
    close(f64(rstd), rr, rr * (rv / 2 + 4 * U))
    h = np.abs(s - rm[:, None]) * rr[:, None]
    tol = np.abs(gn) * (h * (rv[:, None] / 2 + 6 * U) + (rr * dm)[:, None] + rr[:, None] * own) + 2 * U * np.abs(bn) + HALF[dtype] * np.abs(ref)
    close(f64(y), ref, tol * 1.01 + 1e-30)
    if residual:
        close(f64(total), s, (HALF[dtype] + U) * np.abs(s))
    return c, x, r, gain, bias, y, total, mean, rstd


SIZES = [(1, 1), (3, 7), (130, 37), (33, 64), (5, 129), (300, 256), (777, 1024), (17, 1022), (9, 1021), (64, 2048),
         (7, 4100), (3, 8192), (5, 8191), (2, 16384), (3, 16385), (2, 20002), (2, 40960)]


@pytest.mark.parametrize("dtype,params", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,d", SIZES)
def test_forward(T, d, dtype, params, moe_lib, cuda_device):
    check_forward(moe_lib, T, d, dtype, params, False)
    check_forward(moe_lib, T, d, dtype, params, True)


def test_forward_without_parameters(moe_lib, cuda_device):
    check_forward(moe_lib, 50, 96, "bf16", "f32", True, plain=True)
    check_forward(moe_lib, 3, 20000, "f32", "f32", False, plain=True)
    check_forward(moe_lib, 50, 96, "f32", "f32", False, eps=0.1)


def test_forward_far_from_zero(moe_lib, cuda_device):
    """Rows whose mean is a thousand times their spread: squares are of differences."""
    check_forward(moe_lib, 200, 1024, "f32", "f32", False, offset=1000.0)


def test_statistics_may_be_left_out(moe_lib, cuda_device):
    c, x, r, gain, bias, y, total, mean, rstd = check_forward(moe_lib, 70, 128, "bf16", "f32", True)
    y2 = torch.empty_like(y)
    t2 = torch.empty_like(total)
    moe_lib.layer_norm(c, x, gain, bias, y2, residual=r, total=t2)
    assert torch.equal(y, y2) and torch.equal(total, t2)


@pytest.mark.parametrize("d", [96, 1000, 20000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(d, dtype, moe_lib, cuda_device):
    """y or total in the place of x or residual."""
    moe = moe_lib
    c, x, r, gain, bias, y, total, _, _ = check_forward(moe, 40, d, dtype, "f32", True)
    a, b = x.clone(), r.clone()
    moe.layer_norm(c, a, gain, bias, b, residual=b, total=a)
    assert torch.equal(a, total) and torch.equal(b, y)
    a, b = x.clone(), r.clone()
    moe.layer_norm(c, a, gain, bias, a, residual=b, total=b)
    assert torch.equal(b, total) and torch.equal(a, y)
    c, x, _, gain, bias, y, _, _, _ = check_forward(moe, 40, d, dtype, "f32", False)
    moe.layer_norm(c, x, gain, bias, x)
    assert torch.equal(x, y)


@pytest.mark.parametrize("d", [100, 2048, 20000])
def test_rows_that_are_not_finite(d, moe_lib, cuda_device):
    """NaN or an infinity spoils its own row alone; a constant row gives the bias."""
    x, r, gain, bias, dy, dt = make(20, d, "f32", "f32")
    x[3, 5], x[7, d - 1], x[11] = float("nan"), float("inf"), 2.0
    c = moe_lib.make_norm_config(20, d, dtype="f32")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(20, device="cuda"), torch.empty(20, device="cuda")
    moe_lib.layer_norm(c, x, gain, bias, y, mean=mean, rstd=rstd)
    moe_lib.layer_norm_backward(c, dy, x, gain, mean, rstd, dx, None, None, None)
    for t in (y, dx):
        bad = torch.isnan(t).all(dim=1).cpu()
        assert bad.tolist() == [i in (3, 7) for i in range(20)]
        assert torch.isfinite(t[~bad.cuda()]).all()
    assert torch.equal(y[11], bias)


def check_backward(moe, T, d, dtype, params, dtotal, accumulate=False, slack=1.0):
    x, _, gain, _, dy, dt = make(T, d, dtype, params, seed=1)
    c = moe.make_norm_config(T, d, dtype=dtype, param_dtype=params, accumulate=accumulate)
    xs = f64(x)
    _, mean, rstd = O.norm(xs, np.ones(d), np.zeros(d), 1e-5)
    mean_t, rstd_t = torch.tensor(mean).float().cuda(), torch.tensor(rstd).float().cuda()
    mean, rstd = f64(mean_t), f64(rstd_t)
    dx = torch.full_like(x, float("nan"))
    g0 = torch.randn(2, d, generator=torch.Generator().manual_seed(2)).cuda() if accumulate else \
        torch.full((2, d), float("nan"), device="cuda")
    dg, db = g0[0].clone(), g0[1].clone()
    ws = torch.full((moe.norm_workspace_bytes(c),), 0xAB, dtype=torch.uint8, device="cuda")
    moe.layer_norm_backward(c, dy, x, gain, mean_t, rstd_t, dx, dg, db, ws, dtotal=dt if dtotal else None)
    moe.get_error()
    gn, dyn = f64(gain), f64(dy)
    rx, rg, rb = O.norm_backward(dyn, xs, gn, mean, rstd)
    h, g = np.abs((xs - mean[:, None]) * rstd[:, None]), np.abs(dyn * gn)
    rs = rstd[:, None]
    m1, m2 = g.mean(axis=1, keepdims=True), (g * h).mean(axis=1, keepdims=True)
    tol = rs * ((N + 4 * U) * m1 + h * (N + 8 * U) * m2 + 6 * U * (g + m1 + h * m2))
    if dtotal:
        rx = rx + f64(dt)
        tol = tol + 2 * U * np.abs(f64(dt))
    close(f64(dx), rx, tol + HALF[dtype] * np.abs(rx) * 1.01)
    if accumulate:
        rg, rb = rg + f64(g0[0]), rb + f64(g0[1])
    # T terms one after another at the worst, and three roundings of each product
    close(f64(dg), rg, (T + 16) * U * ((np.abs(dyn) * h).sum(axis=0) + np.abs(f64(g0[0]) if accumulate else 0)) + 1e-30)
    close(f64(db), rb, (T + 16) * U * (np.abs(dyn).sum(axis=0) + np.abs(f64(g0[1]) if accumulate else 0)) + 1e-30)
    return c, x, gain, dy, dt, mean_t, rstd_t, dx, dg, db, ws, g0


@pytest.mark.parametrize("dtype,params", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,d", SIZES + [(1500, 64), (1300, 515)])
def test_backward(T, d, dtype, params, moe_lib, cuda_device):
    check_backward(moe_lib, T, d, dtype, params, False)
    check_backward(moe_lib, T, d, dtype, params, True, accumulate=True)


@pytest.mark.parametrize("T,d", [(700, 96), (300, 1024), (40, 20000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_parts(T, d, dtype, moe_lib, cuda_device):
    """Outputs left out, in place of inputs, and again: bit for bit the same."""
    moe = moe_lib
    c, x, gain, dy, dt, mean, rstd, dx, dg, db, ws, _ = check_backward(moe, T, d, dtype, "f32", True)
    a, g2, b2 = torch.empty_like(dx), torch.empty_like(dg), torch.empty_like(db)
    ws.fill_(0xCD)
    moe.layer_norm_backward(c, dy, x, gain, mean, rstd, a, g2, b2, ws, dtotal=dt)
    assert torch.equal(a, dx) and torch.equal(g2, dg) and torch.equal(b2, db)
    moe.layer_norm_backward(c, dy, x, gain, mean, rstd, a.zero_(), None, None, None, dtotal=dt)
    assert torch.equal(a, dx)
    moe.layer_norm_backward(c, dy, x, gain, mean, rstd, None, g2.zero_(), None, ws, dtotal=dt)
    assert torch.equal(g2, dg)
    moe.layer_norm_backward(c, dy, x, gain, mean, rstd, None, None, b2.zero_(), ws)
    assert torch.equal(b2, db)
    for at in range(3):
        t = [dy.clone(), x.clone(), dt.clone()]
        moe.layer_norm_backward(c, t[0], t[1], gain, mean, rstd, t[at], g2.zero_(), b2.zero_(), ws, dtotal=t[2])
        assert torch.equal(t[at], dx) and torch.equal(g2, dg) and torch.equal(b2, db)


def test_gradient_by_differences(moe_lib, cuda_device):
    """Forward and backward together: <dy, y(x + h v) - y(x - h v)> / 2h against <dx, v>, fp32."""
    x, r, gain, bias, dy, v = make(40, 512, "f32", "f32", seed=4)
    c = moe_lib.make_norm_config(40, 512, dtype="f32")

    def y(s):
        out = torch.empty_like(s)
        mean, rstd = torch.empty(40, device="cuda"), torch.empty(40, device="cuda")
        moe_lib.layer_norm(c, s, gain, bias, out, mean=mean, rstd=rstd)
        return out, mean, rstd
    _, mean, rstd = y(x)
    dx = torch.empty_like(x)
    moe_lib.layer_norm_backward(c, dy, x, gain, mean, rstd, dx, None, None, None)
    h = 2.0 ** -6
    up, down = y((x + h * v))[0], y((x - h * v))[0]
    slope = float((dy.double() * (up.double() - down.double())).sum()) / (2 * h)
    want = float((dx.double() * v.double()).sum())
    # h^2 / 6 times third derivatives: of size |dy| |v|^3 per row, and 2^-24 / h of |dy| |y| rounding, summed over
    # 20480 elements as independent errors
    size = float((dy.abs() * v.abs()).double().pow(2).sum()) ** 0.5
    assert abs(slope - want) <= size * (h * h * 10 + 2.0 ** -18)


def test_no_rows(moe_lib, cuda_device):
    c = moe_lib.make_norm_config(0, 40, dtype="f32")
    e, m = torch.empty(0, 40, device="cuda"), torch.empty(0, device="cuda")
    moe_lib.layer_norm(c, e, None, None, e.clone())
    dg, db = torch.ones(40, device="cuda"), torch.ones(40, device="cuda")
    ws = torch.empty(moe_lib.norm_workspace_bytes(c), dtype=torch.uint8, device="cuda")
    moe_lib.layer_norm_backward(c, e, e, None, m, m, e.clone(), dg, db, ws)
    assert (dg == 0).all() and (db == 0).all()
    moe_lib.get_error()


def test_many_rows(moe_lib, cuda_device):
    """More rows than blocks take in one round, and offsets past 2^31 elements."""
    T, d = 1_050_000, 2048
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_()
    c = moe_lib.make_norm_config(T, d)
    y = torch.empty_like(x)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    moe_lib.layer_norm(c, x, None, None, y, mean=mean, rstd=rstd)
    for t in (0, 1, T // 2, T - 2, T - 1):
        ref, rm, rr = O.norm(f64(x[t:t + 1]), 1.0, 0.0, 1e-5)
        close(f64(y[t:t + 1]), ref, np.abs(ref) * HALF["bf16"] * 1.01 + 1e-5)
    dx, dg = torch.empty_like(x), torch.empty(d, device="cuda")
    ws = torch.empty(moe_lib.norm_workspace_bytes(c), dtype=torch.uint8, device="cuda")
    moe_lib.layer_norm_backward(c, x, x, None, mean, rstd, dx, dg, None, ws)
    for t in (0, T // 2, T - 1):
        ref, _, _ = O.norm_backward(f64(x[t:t + 1]), f64(x[t:t + 1]), 1.0, f64(mean[t:t + 1]), f64(rstd[t:t + 1]))
        close(f64(dx[t:t + 1]), ref, np.abs(ref) * HALF["bf16"] * 1.01 + 1e-5)
    del dx, y
    n = (x[:, :64].double() * ((x[:, :64].double() - mean.double()[:, None]) * rstd.double()[:, None])).sum(0)
    # sums of T positive terms near 1: blocks of T / 1216 rows, then 1216 / 8 and 8 partial sums
    assert ((dg[:64].double() - n).abs() <= n * (T / 1216 + 200) * U).all()


def test_other_stream_and_graph(moe_lib, cuda_device):
    moe = moe_lib
    x, r, gain, bias, dy, dt = make(300, 256, "bf16", "f32")
    c = moe.make_norm_config(300, 256)
    cur = torch.zeros_like(x)
    y, total, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(300, device="cuda"), torch.empty(300, device="cuda")
    dg, db = torch.empty(256, device="cuda"), torch.empty(256, device="cuda")
    ws = torch.empty(moe.norm_workspace_bytes(c), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        moe.layer_norm(c, cur, gain, bias, y, residual=r, total=total, mean=mean, rstd=rstd, stream=stream)
        moe.layer_norm_backward(c, dy, total, gain, mean, rstd, dx, dg, db, ws, dtotal=dt, stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    cur.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, total, mean, rstd, dx, dg, db)]
    step()
    for a, b in zip(got, (y, total, mean, rstd, dx, dg, db)):
        assert torch.equal(a, b)
    moe.get_error()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [2, 8, 12, 33, 63, 64, 65, 96, 127, 128])
def test_short_rows(d, dtype, moe_lib, cuda_device):
    """Several rows to a warp: fewer rows than a warp takes, ragged ends, many copies of rows; in place."""
    for T in (1, 3, 31, 1001, 40003):
        check_forward(moe_lib, T, d, dtype, "f32", False)
        c, x, r, gain, bias, y, total, _, _ = check_forward(moe_lib, T, d, dtype, "f32", True)
        moe_lib.layer_norm(c, x, gain, bias, r, residual=r, total=x)
        assert torch.equal(x, total) and torch.equal(r, y)
    check_backward(moe_lib, 1001, d, dtype, "f32", True)
    check_backward(moe_lib, 31, d, dtype, "f32", False)
