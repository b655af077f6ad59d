"""The training-step oracle against independent forms: hand-worked values, central differences
and closed forms. CPU only."""
import math

import numpy as np
import pytest

from oracle import train_oracle as O


def test_embed_hand_worked():
    W = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    ids = np.array([2, 0, 2, -1, 3])
    y = O.embed(ids, W, 0.5)
    assert y.tolist() == [[2.5, 3.0], [0.5, 1.0], [2.5, 3.0], [0.0, 0.0], [0.0, 0.0]]
    dy = np.array([[1.0, 10.0], [2.0, 20.0], [4.0, 40.0], [8.0, 80.0], [16.0, 160.0]])
    dW, _, n = O.embed_backward(ids, dy, 3, 0.5)
    assert dW.tolist() == [[1.0, 10.0], [0.0, 0.0], [2.5, 25.0]] and n.tolist() == [1, 0, 2]
    dW, _, _ = O.embed_backward(ids, dy, 3, 0.5, pad=2, dW0=np.ones((3, 2)))
    assert dW.tolist() == [[2.0, 11.0], [1.0, 1.0], [1.0, 1.0]]


def test_embed_backward_is_the_transpose():
    """<embed(W), dy> = <W, embed_backward(dy)> for every W."""
    rng = np.random.default_rng(0)
    ids, W, dy = rng.integers(0, 7, 40), rng.normal(size=(7, 5)), rng.normal(size=(40, 5))
    assert math.isclose((O.embed(ids, W, 1.5) * dy).sum(), (W * O.embed_backward(ids, dy, 7, 1.5)[0]).sum(),
                        rel_tol=1e-12)


def test_policy_hand_worked():
    """Two tokens of a uniform two-token vocabulary: p = 1/2, one clipped and one not."""
    z = np.zeros((2, 2))
    out = O.policy(z, np.array([0, 1]), np.array([1.0, 1.0]), old=np.log([0.25, 0.5]), w=np.array([1.0, 3.0]))
    # ratio 2 is clipped to 1.2 (no gradient), ratio 1 is not
    assert np.allclose(out["logp"], math.log(0.5)) and math.isclose(out["loss"], -1.2 - 3.0)
    assert (out["dz"][0] == 0).all() and np.allclose(out["dz"][1], [1.5, -1.5])


@pytest.mark.parametrize("kl", [0.0, 0.3])
@pytest.mark.parametrize("on_policy", [False, True])
def test_policy_gradient_against_differences(kl, on_policy):
    rng = np.random.default_rng(1)
    T, V, tau = 12, 9, 0.7
    z, target = rng.normal(size=(T, V)), rng.integers(0, V, T)
    target[3] = -1
    adv, w = rng.normal(size=T), rng.uniform(0.5, 1.5, T)
    w[5] = 0.0
    lp = O.log_softmax_at(z, np.maximum(target, 0), tau)
    old, ref = lp - rng.choice([-0.4, -0.1, 0.1, 0.4], T), lp + rng.normal(size=T) * 0.3
    out = O.policy(z, target, adv, None if on_policy else old, ref, w, tau, 0.2, 0.3, kl)
    if on_policy:      # r is then exp(lp - constant) at that constant = lp
        old = lp
    loss = lambda q: O.policy(q, target, adv, old, ref, w, tau, 0.2, 0.3, kl)["loss"]  # noqa: E731
    h = 1e-6
    for t in range(T):
        for v in range(V):
            up, down = z.copy(), z.copy()
            up[t, v] += h
            down[t, v] -= h
            assert abs((loss(up) - loss(down)) / (2 * h) - out["dz"][t, v]) < 1e-8
    assert (out["dz"][3] == 0).all() and (out["dz"][5] == 0).all()
    assert np.allclose(out["dz"].sum(axis=1), 0, atol=1e-12)       # a softmax gradient sums to zero


def test_adamw_first_step_is_the_sign():
    g = np.array([3.0, -1e-3, 0.0])
    x, m, v, _ = O.adamw(np.ones(3), g, np.zeros(3), np.zeros(3), 1, 0.1, 0.9, 0.999, 1e-12, 0.5)
    assert np.allclose(x, 0.95 - 0.1 * np.sign(g)) and np.allclose(m, 0.1 * g) and np.allclose(v, 1e-3 * g * g)


def test_e4m3_codes_against_torch():
    import torch
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(codes, O.e4m3_values(), equal_nan=True)


def test_dithered_rounding():
    """On the grid, within a step below or above, exact on grid values, right on average."""
    grid = np.sort(O.e4m3_values()[:127])
    rng = np.random.default_rng(2)
    y = np.concatenate([rng.uniform(0, 448, 500), rng.uniform(0, 2.0 ** -5, 500), grid])
    d = rng.integers(0, 1 << 20, len(y)).astype(float)
    q = O.held(y, d, False)
    assert np.isin(q, grid).all()
    below = grid[np.searchsorted(grid, y, "right") - 1]
    above = grid[np.minimum(np.searchsorted(grid, y, "left"), len(grid) - 1)]
    assert ((q == below) | (q == above)).all() and (q[-len(grid):] == grid).all()
    every = np.arange(0, 1 << 20, 64, dtype=float)
    for a in (0.0007, 0.013, 1.03, 77.7, 431.0):
        unit = 2.0 ** max(math.floor(math.log2(a)) - 3, -9)
        assert abs(O.held(np.full(len(every), a), every, False).mean() - a) < unit * 64 / 2 ** 20 * 1.01
    assert O.held(np.array([1e-9, 0.0]), np.zeros(2), True).tolist() == [2.0 ** -9, 0.0]


def test_dither_covers_steps_evenly():
    """Over any run of steps the dither of one element is spread like a golden-ratio sequence."""
    for i in (0, 5, 12345):
        d = np.sort(np.array([O.dither(1, s, start=i)[0] for s in range(1, 257)])) / 2 ** 20
        assert np.diff(d).max() < 3 / 256 and d[0] < 3 / 256 and d[-1] > 1 - 3 / 256
