"""How exact orth(u) is in two-part products (MOE_F32), and every size of cluster that keeps a matrix in shared memory.

The oracle holds operands in two fp16 parts and cuts sums off as the tensor cores do where at most 24 additions go to one
partial sum; kernels stay within twice its distance from the exact result, and 2^-20 for the scale and the sums before
it. What the header says of full-rank matrices, 5e-6, is asked for with a fifth to spare. A part of an operand or a
product of parts that were lost would be 7e-5 at least (the CPU test below)."""
import numpy as np
import pytest
import torch

from oracle import operator_oracle as O

# one cluster of 1 to 8 CTAs (128 of the longer side to each); then tiles
CLUSTERS = [(45, 37), (128, 128), (120, 200), (300, 64), (100, 400), (512, 128), (33, 600), (640, 128), (70, 700), (768, 128), (128, 770),
            (896, 90), (897, 128), (128, 1024)]
TILES = [(257, 2048), (600, 640), (2500, 130), (130, 4000), (300, 300), (35, 1500), (1100, 128)]


def make(rows, cols, seed=1):
    g = torch.Generator().manual_seed(seed)
    r = min(3, rows, cols)
    u = torch.randn(2, rows, cols, generator=g)
    return (u + torch.randn(2, rows, r, generator=g) @ torch.randn(2, r, cols, generator=g)) * 1e-3


def orthogonalize(moe, u, precision):
    n, r, c = u.shape
    cfg = moe.make_muon_config(n, r, c, dtype="f32", grad_dtype="f32", precision=precision)
    ws = torch.full((moe.muon_workspace_bytes(cfg),), 0xFF, dtype=torch.uint8, device="cuda")
    o = torch.full(u.shape, float("nan"), device="cuda")
    moe.orthogonalize(cfg, u.cuda(), o, ws)
    again = torch.empty_like(o)
    moe.orthogonalize(cfg, u.cuda(), again, ws)
    moe.get_error()
    assert torch.equal(o, again)
    return o.double().cpu().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", CLUSTERS + TILES)
def test_full_rank(shape, moe_lib, cuda_device):
    u = make(*shape)
    for precision in ("f32", "bf16"):
        got = orthogonalize(moe_lib, u, precision)
        for i in range(2):
            x = u[i].double().numpy()
            ref = O.orth(x)
            model = O.orth(x, held=O.two_parts()) if precision == "f32" else O.orth_one_part(x)
            err = np.linalg.norm(got[i] - ref) / np.linalg.norm(ref)
            assert err <= 2 * np.linalg.norm(model - ref) / np.linalg.norm(ref) + 2.0 ** -20, (precision, i, err)
            assert err <= (6e-6 if precision == "f32" else 3e-3), (precision, i, err)


@pytest.mark.parametrize("lost", ["X", "A", "B"])
def test_a_lost_part_would_show(lost):
    one, two = O.fp16_planes(1), O.fp16_planes(2)
    for shape in ((257, 300), (45, 37)):
        x = make(*shape)[0].double().numpy()
        ref = O.orth(x)

        def held(v, what):
            return v if isinstance(what, tuple) else (one if what == lost else two)(v, what)
        assert np.linalg.norm(O.orth(x, held=held) - ref) > 10 * 6e-6 * np.linalg.norm(ref)
        bound = 2 * np.linalg.norm(O.orth(x, held=O.two_parts()) - ref) + 2.0 ** -20 * np.linalg.norm(ref)
        assert bound < 2e-5 * np.linalg.norm(ref)
