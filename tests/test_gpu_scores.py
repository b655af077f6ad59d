"""Choice of experts from scores, and its gradient, against the fp64 oracle.

Tolerances count roundings of 2^-24 of a value. x = z / temperature is off by 2 of them, which e^x
turns into 2 |x| relative to it (softmax: of x and of the row's largest); exponential 2, division 2,
sums of up to E = 256 terms in 8 + 5 + 1 additions, the weight's own scale and division 3."""
import numpy as np
import pytest
import torch

from oracle import operator_oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def rel(z, tau):
    """Relative error of a row's scores, by the bound above: [T, 1]."""
    with np.errstate(invalid="ignore"):
        x = np.where(np.isfinite(z), np.abs(z), 0).max(axis=1, keepdims=True) / tau
    return U * (4 * x + 2 + 2 + 14)


def make(T, E, seed=0, std=1.0, bias=True):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=g) * std
    return z, torch.randn(E, generator=g) * 0.05 if bias else None


def run(moe, z, bias, kind, k, groups=1, kept=1, top=1, renorm=True, scale=1.0, tau=1.0):
    T, E = z.shape
    c = moe.make_score_config(T, E, k, score=kind, groups=groups, groups_kept=kept, group_top=top, renormalise=renorm,
                              temperature=tau, scale=scale)
    zc, bc = z.cuda(), None if bias is None else bias.cuda()
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    n = torch.full((E,), -7, dtype=torch.int32, device="cuda")
    bal = torch.full((1,), float("nan"), device="cuda")
    ws = torch.full((moe.route_scores_workspace_bytes(c),), 0xAB, dtype=torch.uint8, device="cuda")
    moe.route_scores(c, zc, bc, idx, w, n, bal, ws)
    i2, w2 = torch.empty_like(idx), torch.empty_like(w)
    moe.route_scores(c, zc, bc, i2, w2)                 # no counts wanted: the same choice, bit for bit
    assert torch.equal(idx, i2) and torch.equal(w.view(torch.int32), w2.view(torch.int32))
    moe.get_error()
    return c, zc, idx, w, n, bal


def check(moe, z, bias, kind, k, groups=1, kept=1, top=1, renorm=True, scale=1.0, tau=1.0, all_rows=False):
    T, E = z.shape
    c, zc, idx, w, n, bal = run(moe, z, bias, kind, k, groups, kept, top, renorm, scale, tau)
    zn, bn, tau = f64(z), None if bias is None else f64(bias), float(np.float32(tau))
    want, s, gap = O.choose(zn, bn, kind, k, groups, kept, top, tau)
    got = idx.cpu().numpy().astype(np.int64)
    r = rel(zn, tau)
    # values this near may stand either way round (scores of 1 at most, a bias of 0.3, sums of two)
    clear = np.ones(T, dtype=bool) if all_rows else gap > 4 * r[:, 0] * (1 + (0 if bias is None else np.abs(bn).max()))
    assert clear.mean() > 0.9
    assert (got[clear] == want[clear]).all()
    for t in range(T):
        assert len(set(got[t])) == k and (got[t] >= 0).all() and (got[t] < E).all()
    ref = O.weights(zn, s, got, kind, renorm, float(np.float32(scale)), tau)
    assert (np.abs(f64(w) - ref) <= np.abs(ref) * (2 * r + (k + 3) * U) + 1e-37).all()
    cn, cb = O.counts(got, E)
    assert (n.cpu().numpy() == cn).all()
    assert abs(float(bal) - cb) <= 2 * U * cb
    return c, zc, idx


GROUPS = [(1, 1, 1), (4, 2, 1), (4, 2, 2), (8, 3, 2)]


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 16, 4), (33, 32, 8), (100, 40, 3), (257, 64, 1), (1000, 128, 8), (999, 200, 8),
                                   (3001, 256, 8)])
def test_choice(T, E, k, kind, with_bias, moe_lib, cuda_device):
    z, bias = make(T, E, bias=with_bias)
    for groups, kept, top in GROUPS:
        if k <= E // groups * kept:
            check(moe_lib, z, bias, kind, k, groups, kept, top)
    check(moe_lib, z, bias, kind, k, renorm=False, scale=2.5, tau=0.7)


@pytest.mark.parametrize("E,groups,kept", [(5, 1, 1), (1, 1, 1), (7, 7, 3), (32, 32, 8), (96, 32, 5), (30, 10, 4),
                                           (255, 5, 2), (256, 2, 1), (256, 16, 1)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_group_shapes(E, groups, kept, kind, moe_lib, cuda_device):
    z, bias = make(300, E, seed=3)
    k = min(8, E // groups * kept)
    for top in (1, 2):
        check(moe_lib, z, bias, kind, k, groups, kept, top)
        check(moe_lib, z, None, kind, k, groups, kept, top, renorm=k > 1)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept,top", GROUPS)
def test_exact_ties(kind, groups, kept, top, moe_lib, cuda_device):
    """Small whole logits and biases: equal values tie exactly on both sides, others are far apart."""
    g = torch.Generator().manual_seed(5)
    z = torch.randint(0, 3, (400, 64), generator=g).float()
    check(moe_lib, z, None, kind, 8, groups, kept, 1, all_rows=True)
    if kind == "sigmoid":       # s + b: 0.5, 0.731, 0.881 with 0 or 2 added; equal only where both are equal
        bias = torch.randint(0, 2, (64,), generator=g).float() * 2
        check(moe_lib, z, bias, kind, 8, groups, kept, 1, all_rows=True)
    check(moe_lib, torch.zeros(40, 256), None, kind, 8, all_rows=True)      # every expert ties
    check(moe_lib, torch.zeros(40, 256), torch.zeros(256), kind, 8, 8, 3, 2, all_rows=True)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked_experts(kind, with_bias, moe_lib, cuda_device):
    """Logits of -inf: taken last, with weight 0; rows that hold nothing else."""
    z, bias = make(200, 48, seed=6, bias=with_bias)
    g = torch.Generator().manual_seed(7)
    z[torch.rand(200, 48, generator=g) < 0.8] = float("-inf")
    z[:20] = float("-inf")
    z[20:30, 1:] = float("-inf")
    low = torch.finfo(torch.float32).min
    for renorm in (True, False):
        c, zc, idx, w, n, _ = run(moe_lib, z, bias, kind, 8, renorm=renorm)
        got, wn = idx.cpu().numpy().astype(np.int64), f64(w)
        want, s, gap = O.choose(f64(z), None if bias is None else f64(bias), kind, 8)
        clear = gap > 1e-5
        assert (got[clear] == want[clear]).all()
        taken = np.take_along_axis(f64(z), got, axis=1)
        assert (wn[np.isneginf(taken)] == 0).all() and np.isfinite(wn).all()
        assert (got[:20] == np.arange(8)).all() and (wn[:20] == 0).all()
        assert (got[20:30, 0] == 0).all()
        if renorm:
            # one expert is left in rows 20 to 29, none where the draw above has masked that one too
            assert np.abs(wn[20:30, 0] - torch.isfinite(z[20:30, 0]).numpy()).max() < 1e-6
    z[torch.isinf(z)] = low                               # the type's lowest value instead
    _, _, idx, w, _, _ = run(moe_lib, z, bias, kind, 8)
    got, wn = idx.cpu().numpy(), f64(w)
    assert np.isfinite(wn).all() and all(len(set(r)) == 8 for r in got)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(E, g) for E in (32, 64, 128, 256) for g in (2, 4, 8, 16, 32)])
def test_groups_of_whole_rows(E, groups, kind, moe_lib, cuda_device):
    """Rows of whole registers, groups of one expert to half a row: random values, equal ones, masked ones."""
    kept = max(1, groups // 4)
    k = min(8, E // groups * kept)
    z, bias = make(211, E, seed=E + groups)
    for top in (1, 2):
        check(moe_lib, z, bias, kind, k, groups, kept, top, renorm=k > 1)
    g = torch.Generator().manual_seed(E * groups)
    few = torch.randint(0, 9, (211, E), generator=g).float()       # whole numbers tie exactly on both sides
    check(moe_lib, few, None, kind, k, groups, kept, 1, renorm=k > 1, all_rows=True)
    few[torch.rand(211, E, generator=g) < 0.9] = float("-inf")     # open groups with fewer than k, or none
    few[:5] = float("-inf")
    _, _, idx, w, _, _ = run(moe_lib, few, None, kind, k, groups, kept, 1)
    want, _, _ = O.choose(f64(few), None, kind, k, groups, kept, 1)
    got = idx.cpu().numpy().astype(np.int64)
    assert (got == want).all()
    assert (f64(w)[np.isneginf(np.take_along_axis(f64(few), got, axis=1))] == 0).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept,top", GROUPS)
def test_rows_that_are_not_finite(kind, groups, kept, top, moe_lib, cuda_device):
    z, bias = make(64, 64, seed=8)
    z[3, 5], z[10, 60], z[20] = float("nan"), float("inf"), float("nan")
    for b in (None, bias):
        _, _, idx, w, _, _ = run(moe_lib, z, b, kind, 8, groups, kept, top)
        got, wn = idx.cpu().numpy(), f64(w)
        assert all(len(set(r)) == 8 for r in got) and (got >= 0).all() and (got < 64).all()
        want, _, gap = O.choose(f64(z), None if b is None else f64(b), kind, 8, groups, kept, top)
        bad = {3, 10, 20} if kind == "softmax" else {20}
        for t in range(64):
            assert np.isnan(wn[t]).all() == (t in bad), t
            if gap[t] > 1e-4:
                assert (got[t] == want[t]).all(), t
        if kind == "sigmoid":
            assert 5 not in got[3] and got[10, 0] == 60 or groups > 1


def test_far_scores(moe_lib, cuda_device):
    """Logits so far apart that scores round to 0 or 1: the order is still that of the logits."""
    z = torch.linspace(-300, 300, 64).repeat(5, 1)[:, torch.randperm(64, generator=torch.Generator().manual_seed(1))]
    for kind in ("softmax", "sigmoid"):
        _, _, idx, w, _, _ = run(moe_lib, z, None, kind, 8)
        assert torch.equal(idx.cpu().long(), z.topk(8).indices)
        assert torch.isfinite(w).all()
    _, _, idx, w, _, _ = run(moe_lib, -z.abs() - 200, None, "sigmoid", 8)     # every score is 0 in fp32
    assert (w == 0).all()


def grad(moe, c, z, idx, dw):
    dz = torch.full(z.shape, float("nan"), device="cuda")
    moe.route_scores_backward(c, z, idx, dw, dz)
    moe.get_error()
    return dz


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 4, 1), (2, 7, 3), (3, 33, 8), (66, 64, 2), (1001, 45, 5), (1000, 128, 8),
                                   (2050, 256, 8), (777, 201, 7)])
def test_gradient(T, E, k, kind, renorm, moe_lib, cuda_device):
    z, bias = make(T, E, seed=9)
    tau, scale = 0.7, 2.5
    c, zc, idx = check(moe_lib, z, bias, kind, k, renorm=renorm, scale=scale, tau=tau)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(1)).cuda()
    got = f64(grad(moe_lib, c, zc, idx, dw))
    tau = float(np.float32(tau))
    i = idx.cpu().numpy().astype(np.int64)
    ref, size = O.scores_backward(f64(z), i, f64(dw), kind, renorm, float(np.float32(scale)), tau)
    # scores, shares and slope each as in rel(), and k + 5 more operations
    assert (np.abs(got - ref) <= size * (4 * rel(f64(z), tau) + (k + 5) * U)).all()
    if kind == "sigmoid" or renorm:
        rest = np.ones((T, E), dtype=bool)
        np.put_along_axis(rest, i, False, axis=1)
        assert (got[rest] == 0).all()


def test_gradient_where_one_share_is_all(moe_lib, cuda_device):
    """Shares of nearly one: the others' tiny gradients come by differences, without cancelling."""
    z = torch.zeros(8, 16)
    z[:, 3], z[:, 7] = 20.0, 4.0
    for kind in ("softmax", "sigmoid"):
        c, zc, idx = check(moe_lib, z * (1 if kind == "softmax" else -1), None, kind, 3, all_rows=True)
        dw = torch.tensor([[1.0, 0.5, -0.25]]).repeat(8, 1).cuda()
        got = f64(grad(moe_lib, c, zc, idx, dw))
        zn = f64(zc)
        ref, size = O.scores_backward(zn, idx.cpu().numpy().astype(np.int64), f64(dw), kind, True, 1.0, 1.0)
        assert (np.abs(got - ref) <= size * (4 * rel(zn, 1.0) + 8 * U)).all()


@pytest.mark.parametrize("kind,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gradient_of_bad_rows(kind, renorm, moe_lib, cuda_device):
    """Experts out of range or named twice are left out and reported; -inf logits have no gradient."""
    moe = moe_lib
    z = torch.randn(6, 20, generator=torch.Generator().manual_seed(2))
    z[4, :] = float("-inf")
    z[5, 2] = float("-inf")
    idx = torch.tensor([[0, 1, 2], [3, 20, 4], [5, 6, 5], [7, -1, 8], [0, 1, 2], [2, 3, 4]], dtype=torch.int32)
    dw = torch.randn(6, 3, generator=torch.Generator().manual_seed(3))
    c = moe.make_score_config(6, 20, 3, score=kind, renormalise=renorm)
    dz = torch.full((6, 20), float("nan"), device="cuda")
    moe.route_scores_backward(c, z.cuda(), idx.cuda(), dw.cuda(), dz)
    with pytest.raises(moe.MoeError) as e:
        moe.get_error()
    assert e.value.status == moe.MOE_ERR_DEVICE_BOUNDS
    got = f64(dz)
    assert np.isfinite(got).all() and (got[4] == 0).all() and got[5, 2] == 0
    for t, slots in ((0, [0, 1, 2]), (1, [0, 2]), (2, [0, 1]), (3, [0, 2]), (5, [0, 1, 2])):
        i = idx[t:t + 1, slots].numpy().astype(np.int64)
        ref, size = O.scores_backward(f64(z[t:t + 1]), i, f64(dw[t:t + 1, slots]), kind, renorm, 1.0, 1.0)
        assert (np.abs(got[t:t + 1] - ref) <= size * (4 * rel(f64(z[t:t + 1]), 1.0) + 8 * U)).all(), t


def test_no_tokens(moe_lib, cuda_device):
    c = moe_lib.make_score_config(0, 16, 4)
    n = torch.full((16,), 5, dtype=torch.int32, device="cuda")
    bal = torch.ones(1, device="cuda")
    ws = torch.empty(moe_lib.route_scores_workspace_bytes(c), dtype=torch.uint8, device="cuda")
    moe_lib.route_scores(c, torch.empty(0, 16, device="cuda"), None, torch.empty(0, 4, dtype=torch.int32, device="cuda"),
                         torch.empty(0, 4, device="cuda"), n, bal, ws)
    assert (n == 0).all() and float(bal) == 0
    moe_lib.get_error()


def test_other_stream_and_graph(moe_lib, cuda_device):
    """A choice and its gradient captured on a side stream, replayed on new logits."""
    moe = moe_lib
    z, bias = make(500, 64, seed=11)
    c = moe.make_score_config(500, 64, 4, score="sigmoid", groups=4, groups_kept=2, group_top=2, scale=2.0)
    zc, bc = torch.zeros_like(z).cuda(), bias.cuda()
    idx, w = torch.empty(500, 4, dtype=torch.int32, device="cuda"), torch.empty(500, 4, device="cuda")
    n, bal = torch.empty(64, dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda")
    dz = torch.empty_like(zc)
    ws = torch.empty(moe.route_scores_workspace_bytes(c), dtype=torch.uint8, device="cuda")
    dw = torch.randn(500, 4, device="cuda")

    def step(stream=None):
        moe.route_scores(c, zc, bc, idx, w, n, bal, ws, stream=stream)
        moe.route_scores_backward(c, zc, idx, dw, dz, stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    zc.copy_(z)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (idx, w, n, bal, dz)]
    step()
    torch.cuda.synchronize()
    for a, b in zip(got, (idx, w, n, bal, dz)):
        assert torch.equal(a, b)
    assert int(n.sum()) == 2000
    moe.get_error()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [100, 128])
def test_bias_that_is_not_finite(E, kind, moe_lib, cuda_device):
    """A bias of NaN counts as one of -inf; one of +inf is chosen first, unless its logit is -inf."""
    z, bias = make(77, E, seed=12)
    bias[3], bias[40], z[5, 40] = float("nan"), float("inf"), float("-inf")
    _, _, idx, w, _, _ = run(moe_lib, z, bias, kind, 8)
    bias[3] = float("-inf")
    _, _, i2, w2, _, _ = run(moe_lib, z, bias, kind, 8)
    assert torch.equal(idx, i2) and torch.equal(w, w2)
    got = idx.cpu().numpy()
    assert (got != 3).all() and (np.delete(got[:, 0], 5) == 40).all() and (got[5] != 40).all()
