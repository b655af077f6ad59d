"""orth(u) where u is not of full rank: the gradient of an expert that few tokens reached, whose rank is theirs
at most. What a rounding leaves in directions that u does not have is multiplied by a = 3.4445 with every step that
follows, so that full-rank noise says nothing of it.

The oracle takes the kernels' roundings in 64 bits; a second set of roundings of that size is off by as much, so the
kernels stay within twice its distance from the exact result. On top of that stands what the header promises for
one-part products: 3e-3 of the result (in rows of less than 16, which average nothing out: 6e-3).
"""
import numpy as np
import pytest
import torch

from oracle import operator_oracle as O

pytestmark = pytest.mark.gpu

SHAPES = [(45, 37), (24, 200), (128, 128), (128, 1000), (1000, 70), (129, 129), (300, 520), (520, 300), (257, 2048),
          (35, 1500), (1500, 40)]


def low_rank(rows, cols, kind, seed):
    """Two matrices: of rank 1, 2, a quarter or half of the side; of a few rows alone; of falling singular values; a
    momentum of 20 gradients of rank 8."""
    g = torch.Generator().manual_seed(seed)
    side = min(rows, cols)

    def product(r):
        return torch.randn(2, rows, r, generator=g, dtype=torch.float64) @ torch.randn(2, r, cols, generator=g, dtype=torch.float64)
    if kind == "three rows":
        u = product(1)
        u[:, 3:] = 0
    elif kind == "falling":
        left, right = (torch.linalg.qr(torch.randn(2, n, side, generator=g, dtype=torch.float64))[0] for n in (rows, cols))
        u = (left * torch.logspace(0, -5, side, dtype=torch.float64)) @ right.mT
    elif kind == "momentum":
        u = sum(0.95 ** i * product(min(8, side)) for i in range(20))
    else:
        u = product(max(1, kind if isinstance(kind, int) else int(kind[0] * side)))
    return (u * 1e-3).float()


KINDS = [1, 2, (0.25,), (0.5,), "three rows", "falling", "momentum"]


def orthogonalize(moe, u, precision):
    n, r, c = u.shape
    cfg = moe.make_muon_config(n, r, c, dtype="f32", grad_dtype="f32", precision=precision)
    ws = torch.full((moe.muon_workspace_bytes(cfg),), 0xFF, dtype=torch.uint8, device="cuda")
    o = torch.full(u.shape, float("nan"), device="cuda")
    moe.orthogonalize(cfg, u.cuda(), o, ws)
    moe.get_error()
    return o.double().cpu().numpy()


def size(x):
    return np.sqrt((x * x).sum())


@pytest.mark.parametrize("kind", KINDS, ids=str)
@pytest.mark.parametrize("shape", SHAPES)
def test_low_rank(shape, kind, moe_lib, cuda_device):
    u = low_rank(*shape, kind, seed=sum(shape))
    for precision in ("bf16", "f32"):
        got = orthogonalize(moe_lib, u, precision)
        for i in range(2):
            x = u[i].double().numpy()
            ref = O.orth(x)
            model = O.orth_one_part(x) if precision == "bf16" else O.orth(x, held=O.two_parts())
            err = size(got[i] - ref) / size(ref)
            # the scale's own rounding, and the sums' before it: 2^-20, as in the tests of full-rank matrices
            assert err <= 2 * size(model - ref) / size(ref) + 2.0 ** -20, (precision, i, err)
            if precision == "bf16":
                assert err <= 3e-3, (i, err)


@pytest.mark.parametrize("shape", [(1, 40), (3, 700), (9, 5), (2, 2000)])
def test_few_rows(shape, moe_lib, cuda_device):
    for kind in (1, 2, "falling"):
        u = low_rank(*shape, min(kind, min(shape)) if isinstance(kind, int) else kind, seed=5)
        got = orthogonalize(moe_lib, u, "bf16")
        for i in range(2):
            ref = O.orth(u[i].double().numpy())
            assert size(got[i] - ref) <= 6e-3 * size(ref), (kind, i)


@pytest.mark.parametrize("shape", [(3, 40, 72), (2, 264, 160), (2, 160, 264)])
@pytest.mark.parametrize("master", [False, True])
def test_step_on_low_rank_gradients(shape, master, moe_lib, cuda_device):
    """A step on bf16 weights by the default precision: what it moves them by, to 3e-3 of its size and the rounding
    of the weights (none of them, with masters)."""
    g = torch.Generator().manual_seed(11)
    n, r, c = shape
    grad = (torch.randn(n, r, 4, generator=g) @ torch.randn(n, 4, c, generator=g) * 1e-3).bfloat16()
    p = (torch.randn(shape, generator=g) * 0.02).bfloat16()
    t = dict(p=p.cuda(), g=grad.cuda())
    if master:
        t["master"] = p.float().cuda()
    moe_lib.Muon([t], lr=0.02, momentum=0.0, nesterov=False).step()
    moe_lib.get_error()
    got = (t["master"] if master else t["p"]).double().cpu().numpy()
    move = 0.02 * 0.2 * np.sqrt(max(r, c))
    for i in range(n):
        ref = O.orth(grad[i].double().numpy())
        want = p[i].double().numpy() - move * ref
        err = np.abs(got[i] - want)
        out = (2.0 ** -24 * 4 if master else 2.0 ** -8 * 1.01) * np.maximum(np.abs(want), np.abs(p[i].double().numpy()))
        assert size(np.maximum(err - out, 0)) <= 3e-3 * move * size(ref), i
