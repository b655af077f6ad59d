"""The lowest temperatures: logits are compared as scores of log2(e) / temperature, which fp32 has to hold."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import operator_oracle as O

LEAST = np.float32(1.4426950408889634 / float(np.finfo(np.float32).max))       # log2(e) over the largest number
LEAST = LEAST if 1.4426950408889634 / float(LEAST) <= float(np.finfo(np.float32).max) else np.nextafter(LEAST, np.float32(1))


@pytest.mark.parametrize("temperature", [2.938737e-39, 3e-39, 3.5e-39, 4.2e-39, float(np.nextafter(LEAST, np.float32(0)))])
def test_refused(temperature, moe_lib):
    """1 / temperature is finite from 2.94e-39 on, log2(e) / temperature from 4.24e-39."""
    lib, P, R = moe_lib.load(), ctypes.c_void_p(256), ctypes.c_void_p(512)
    with np.errstate(over="ignore"):
        assert np.isfinite(np.float32(1) / np.float32(temperature))
    c = moe_lib.make_score_config(10, 16, 4, temperature=temperature)
    assert c.temperature > 0
    assert lib.moe_route_scores_workspace_bytes(ctypes.byref(c)) == 0
    assert lib.moe_route_scores(ctypes.byref(c), P, P, P, P, P, P, P, None) == -1
    assert lib.moe_route_scores_backward(ctypes.byref(c), P, P, P, R, None) == -1
    layer = moe_lib.make_config(10, 64, 16, 4, 64)
    assert lib.moe_backward_scores(ctypes.byref(layer), ctypes.byref(c), P, R, *[P] * 25, None) == -1


@pytest.mark.parametrize("temperature", [float(LEAST), 5e-39, 1.2e-38, 1.0, 3e38])
def test_taken(temperature, moe_lib):
    c = moe_lib.make_score_config(10, 16, 4, temperature=temperature)
    assert moe_lib.route_scores_workspace_bytes(c) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("temperature", [float(LEAST), 5e-39, 1.2e-38])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept,k", [(40, 1, 1, 8), (256, 8, 2, 8), (256, 32, 1, 8), (45, 5, 1, 8), (8, 1, 1, 8)])
def test_choice_at_the_lowest(E, groups, kept, k, kind, temperature, moe_lib, cuda_device):
    """Scores are 0 or 1 there (a half for a sigmoid of 0), and the bias tells their order; without one, logits do."""
    moe, T = moe_lib, 70
    g = torch.Generator().manual_seed(E)
    z = torch.randn(T, E, generator=g)
    z[4, 1:] = float("-inf")
    if E != 45:                      # (its 1 / E is not exact, so that sums of two tie by their rounding)
        z[3] = 0
    bias = (torch.randperm(E, generator=g) - E // 2).float() * 2.0 ** -10
    for b in (None, bias):
        top = 1 if b is None else 2
        c = moe.make_score_config(T, E, k, score=kind, groups=groups, groups_kept=kept, group_top=top, temperature=temperature)
        idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
        w = torch.full((T, k), float("nan"), device="cuda")
        n = torch.full((E,), -7, dtype=torch.int32, device="cuda")
        ws = torch.empty(moe.route_scores_workspace_bytes(c), dtype=torch.uint8, device="cuda")
        moe.route_scores(c, z.cuda(), None if b is None else b.cuda(), idx, w, counts=n, ws=ws)
        moe.get_error()
        want, _, _ = O.choose(z.double().numpy(), None if b is None else b.double().numpy(), kind, k, groups, kept, top,
                              c.temperature)
        got = idx.cpu().numpy()
        assert (got == want).all()
        assert (n.cpu().numpy() == O.counts(got, E)[0]).all()
        assert torch.isfinite(w).all()
