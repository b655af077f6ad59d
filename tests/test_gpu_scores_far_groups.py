"""Groups by the sum of two scores, without a bias: experts in the open groups are told apart by their logits, however
alike their scores round. The logits are such that all groups but the first are worth the same in fp32 (sigmoids that
round to 1; softmax shares that round to 0), so that the lowest stay open and the rest is exact."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

SHAPES = [(256, 8, 4, 8), (256, 32, 3, 8), (256, 2, 1, 5), (128, 4, 2, 8), (64, 8, 2, 3), (32, 4, 1, 8), (45, 5, 2, 7), (160, 8, 4, 8),
          (192, 8, 4, 8), (20, 4, 3, 8), (96, 3, 1, 6)]


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept,k", SHAPES)
def test_order_of_logits(E, groups, kept, k, kind, moe_lib, cuda_device):
    T, size = 333, E // groups
    g = torch.Generator().manual_seed(E + groups)
    z = torch.rand(T, E, generator=g) * 10
    if kind == "sigmoid":
        z += 30                                        # 1 - s < 1e-13
    else:
        z -= 200                                       # e^-190 is 0 in fp32
        z[:, 1] = 0                                    # the largest: the first group is worth 1
        z[::3, 0] = float("-inf")
    c = moe_lib.make_score_config(T, E, k, score=kind, groups=groups, groups_kept=kept, group_top=2)
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    moe_lib.route_scores(c, z.cuda(), None, idx, w)
    moe_lib.get_error()
    want = np.argsort(-z[:, :kept * size].numpy(), axis=1, kind="stable")[:, :k]
    assert (idx.cpu().numpy() == want).all()


def test_rows_without_a_distribution(moe_lib, cuda_device):
    """NaN and infinities, as in any other choice: a sigmoid's NaN is never ahead, a softmax row's experts are the first."""
    T, E, nan, inf = 4, 64, float("nan"), float("inf")
    z = torch.full((T, E), -1.0)
    z[0, 5], z[0, 9], z[0, 11] = nan, 3.0, 2.0
    z[1, 17], z[1, 60] = inf, 8.0
    z[2] = -inf
    z[3, 40:44] = torch.tensor([50.0, 51.0, 53.0, 52.0])
    want = {"sigmoid": [[9, 11, 0], [17, 60, 16], [0, 1, 2], [42, 43, 41]],
            "softmax": [[0, 1, 2], [0, 1, 2], [0, 1, 2], [42, 43, 41]]}
    for kind in want:
        c = moe_lib.make_score_config(T, E, 3, score=kind, groups=4, groups_kept=2, group_top=2)
        idx = torch.full((T, 3), -7, dtype=torch.int32, device="cuda")
        w = torch.empty(T, 3, device="cuda")
        moe_lib.route_scores(c, z.cuda(), None, idx, w)
        moe_lib.get_error()
        assert idx.cpu().tolist() == want[kind]
