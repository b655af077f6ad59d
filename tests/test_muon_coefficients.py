"""Coefficients that fp16 operands do not hold are refused; those just inside give what the formula says."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import operator_oracle as O

USUAL = (3.4445, -4.7750, 2.0315)
# (coefficients, steps): a singular value in [0, 1] brings X or A above 31.9, or b A + c A A above 63.8
REFUSED = [((16, 0, 0), 2), ((2, 0, 0), 7), ((16, 16, 16), 1), ((5.8, 0, 0), 2), ((16, 16, 0), 1), ((-16, -16, 0), 1),
           ((0, 8, 8), 2), ((3.4445, -4.7750, 16), 2), ((1, 5, 0), 2), ((4, -16, 16), 4), ((2, 0, 0), 100)]
TAKEN = [((16, 0, 0), 1), ((5.5, 0, 0), 2), ((0, 0, 0), 100), ((3, 8, 8), 1), ((16, 15.5, 0), 1), ((-5, 0.5, -1), 1), ((16, -16, 0), 1),
         ((1, 0, 0), 100), ((1.5, -0.5, 0), 100), ((1.875, -1.25, 0.375), 100), (USUAL, 100), ((2, -1.5, 0.5), 30), ((16, 16, 16), 0),
         ((4, -16, 16), 1)]


def largest(coef, steps):
    """Largest of X and A, and of b A + c A A, over singular values in [0, 1], from a fine grid."""
    a, b, c = coef
    s, most_x, most_b = 1.0, 1.0, 0.0
    for _ in range(steps):
        g = np.linspace(0, s, 20001)
        most_x, most_b = max(most_x, s * s), max(most_b, np.abs(b * g ** 2 + c * g ** 4).max())
        s = np.abs(g * (a + b * g ** 2 + c * g ** 4)).max()
        most_x = max(most_x, s)
        if most_x > 1e6:
            break
    return most_x, most_b


def config(moe, coef, steps, shape=(2, 64, 32), precision="f32"):
    return moe.make_muon_config(*shape, dtype="f32", precision=precision, coef=coef, steps=steps)


@pytest.mark.parametrize("precision", ["bf16", "f32"])
@pytest.mark.parametrize("coef,steps", REFUSED)
def test_refused(coef, steps, precision, moe_lib):
    x, b = largest(coef, steps)
    assert x > 31.9 or b > 63.8
    lib, P = moe_lib.load(), ctypes.c_void_p(256)
    for shape in ((2, 64, 32), (1, 300, 400), (1, 1, 1)):
        c = config(moe_lib, coef, steps, shape, precision)
        assert moe_lib.muon_workspace_bytes(c) == 0
        assert lib.moe_orthogonalize(ctypes.byref(c), P, P, P, None) == -2
        assert lib.moe_muon(ctypes.byref(c), *[P] * 7, None) == -2
    p = torch.zeros(8, 4)
    with pytest.raises(moe_lib.MoeError) as e:
        moe_lib.Muon([dict(p=p, g=p.clone())], coef=coef, steps=steps)
    assert e.value.status == -2


@pytest.mark.parametrize("coef,steps", TAKEN)
def test_taken(coef, steps, moe_lib):
    x, b = largest(coef, steps)
    assert x < 31.9 and b < 63.8
    assert moe_lib.muon_workspace_bytes(config(moe_lib, coef, steps)) > 0


def test_the_border_is_where_the_grid_says(moe_lib):
    """Random coefficients: refused above the border, taken 1% (and a slack of 2^-9 a step) below it."""
    rng = np.random.default_rng(3)
    seen = [0, 0]
    for _ in range(4000):
        coef, steps = tuple(float(v) for v in rng.uniform(-1, 1, 3) * 16 ** rng.uniform(-1, 1)), int(rng.integers(1, 5))
        x, b = largest(coef, steps)
        size = moe_lib.muon_workspace_bytes(config(moe_lib, coef, steps))
        if x > 31.95 or b > 63.9:
            assert size == 0, (coef, steps)
            seen[0] += 1
        # a step multiplies a slack of 2^-9 by up to |a| + 3 |b| s^2 + 5 |c| s^4 over its result: half is far inside
        elif x < 4 and b < 8:
            assert size > 0, (coef, steps)
            seen[1] += 1
    assert min(seen) > 300


@pytest.mark.gpu
@pytest.mark.parametrize("coef,steps", [((16, 0, 0), 1), ((5.5, 0, 0), 2), ((3, 8, 8), 1), ((16, 15.5, 0), 1), ((4, -16, 16), 1)])
@pytest.mark.parametrize("shape", [(1, 1), (40, 50), (200, 300), (300, 200)])
def test_just_inside(shape, coef, steps, moe_lib, cuda_device):
    """One element alone (a singular value of 1) and random factors: nothing overflows. Without b and c only X's 22
    bits and the scale's rounding (2^-20, as in the other tests) are left; with them the oracle's roundings, twice."""
    g = torch.Generator().manual_seed(2)
    u = torch.zeros(3, *shape)
    u[0, shape[0] - 1, shape[1] // 2] = 3e-4
    u[1:] = torch.randn(2, *shape, generator=g)
    u[2] = torch.randn(shape[0], 1, generator=g) @ torch.randn(1, shape[1], generator=g)
    for precision in ("bf16", "f32"):
        c = config(moe_lib, coef, steps, (3, *shape), precision)
        ws = torch.empty(moe_lib.muon_workspace_bytes(c), dtype=torch.uint8, device="cuda")
        o = torch.full((3, *shape), float("nan"), device="cuda")
        moe_lib.orthogonalize(c, u.cuda(), o, ws)
        moe_lib.get_error()
        for i in range(3):
            x = u[i].double().numpy()
            ref = O.orth(x, steps, coef)
            model = O.orth_one_part(x, steps, coef) if precision == "bf16" else O.orth(x, steps, coef, held=O.two_parts())
            off = 0 if coef[1] == coef[2] == 0 else 2 * np.linalg.norm(model - ref)
            err = np.linalg.norm(o[i].double().cpu().numpy() - ref)
            assert err <= off + 2.0 ** -19 * max(np.linalg.norm(ref), 1), (precision, i, err, off)
