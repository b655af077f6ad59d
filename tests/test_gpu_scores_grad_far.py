"""The softmax's gradient does not depend on what all logits have in common, as its weights do not.

z - max is rounded by 2^-24 of itself, its quotient by 3 (temperature's reciprocal in two parts), e^x turns that into
4 |x - max| 2^-24; exponential 2, sum of up to 256 terms 14, division, scale and temperature 5; a share enters twice,
and the sum over slots adds 8 terms: 2 (4 |x - max| + 21) + 9 roundings of 2^-24 of the terms' size. Where a logit was added
to, its own rounding is in the input and none of the call's."""
import numpy as np
import pytest
import torch

from oracle import operator_oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("offset,tau", [(0.0, 0.7), (1000.0, 0.7), (-5000.0, 0.3), (3e4, 1.3)])
@pytest.mark.parametrize("T,E,k", [(1, 16, 4), (130, 45, 3), (257, 128, 8), (64, 256, 8)])
def test_common_offset(T, E, k, offset, tau, renorm, moe_lib, cuda_device):
    g = torch.Generator().manual_seed(T + E)
    z = (torch.randn(T, E, generator=g) + offset)
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    dw = torch.randn(T, k, generator=g)
    c = moe_lib.make_score_config(T, E, k, score="softmax", renormalise=renorm, temperature=tau, scale=2.5)
    dz = torch.full((T, E), float("nan"), device="cuda")
    moe_lib.route_scores_backward(c, z.cuda(), idx.cuda(), dw.cuda(), dz)
    moe_lib.get_error()
    zn, tau = z.double().numpy(), c.temperature
    want, size = O.scores_backward(zn, idx.numpy(), dw.double().numpy(), "softmax", renorm, 2.5, tau)
    far = (zn.max(1) - zn.min(1))[:, None] / tau
    assert (np.abs(dz.double().cpu().numpy() - want) <= (2 * (4 * far + 21) + 9) * U * size + 1e-37).all()


@pytest.mark.parametrize("renorm", [True, False])
def test_quotients_beyond_fp32(renorm, moe_lib, cuda_device):
    """z / temperature passes fp32; differences of logits are what counts: a lone largest has all of the weight (and no
    gradient), equal ones share it."""
    T, E, k = 40, 24, 3
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(1)) + 300
    z[::2, 3] = z[::2, 7] = 400
    z[1::2, 3] = 400
    idx = torch.tensor([[3, 7, 5]], dtype=torch.int32).repeat(T, 1)
    dw = torch.tensor([[1.0, -1.0, 0.5]]).repeat(T, 1)
    tau = 2.0 ** -120
    c = moe_lib.make_score_config(T, E, k, score="softmax", renormalise=renorm, temperature=tau)
    w, dz = torch.empty(T, k, device="cuda"), torch.full((T, E), float("nan"), device="cuda")
    moe_lib.route_scores_backward(c, z.cuda(), idx.cuda(), dw.cuda(), dz)
    moe_lib.get_error()
    want = torch.zeros(T, E)
    want[::2, 3], want[::2, 7] = 0.5 / tau, -0.5 / tau       # share (dw - mean dw) / tau, exact
    assert torch.equal(dz.cpu(), want)
