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


@pytest.mark.parametrize("root", [False, True])
def test_dithered_rounding(root):
    """On the grid, a neighbour below or above, exact on grid values, and right on average over the
    dither: in the value itself, or in its square."""
    grid = np.sort(O.e4m3_values()[:121])                     # up to 256
    rng = np.random.default_rng(2)
    y = np.concatenate([rng.uniform(0, 256, 500), rng.uniform(2.0 ** -8, 2.0 ** -5, 500), grid])
    d = rng.integers(0, 1 << 20, len(y)).astype(float)
    q = O.held(y, d, root)
    assert np.isin(q, grid).all()
    below = grid[np.searchsorted(grid, y, "right") - 1]
    above = grid[np.minimum(np.searchsorted(grid, y, "left"), len(grid) - 1)]
    assert ((q == below) | (q == above)).all() and (q[-len(grid):] == grid).all()
    every = np.arange(0, 1 << 20, 64, dtype=float)
    k = 2 if root else 1
    for a in (0.0057, 0.013, 1.03, 77.7, 231.0):
        unit = 2.0 ** max(math.floor(math.log2(a)) - 3, -9)
        slack = ((a + unit) ** k - (a - unit) ** k) * 64 / 2 ** 20
        assert abs((O.held(np.full(len(every), a), every, root) ** k).mean() - a ** k) < slack
    assert O.held(np.array([1e-9, 0.0]), np.zeros(2), True).tolist() == [2.0 ** -9, 0.0]


def test_dither_is_even_and_unrelated():
    """Over elements at a step, over steps at an element, and between the two states: uniform to the
    spread of N draws, and uncorrelated (N = 4096: 4 / sqrt(N) is 0.06)."""
    rows = [O.dither(4096, 17), O.dither(4096, 18)]
    cols = [np.array([O.dither(1, s, start=i) for s in range(1, 4097)])[:, :, 0].T for i in (0, 12345)]
    for m, v in rows + [tuple(c) for c in cols]:
        for d in (m, v):
            assert abs(np.bincount((d / 2 ** 16).astype(int), minlength=16) - 256).max() < 5 * 16
        for a, b in ((m, v), (m[1:], m[:-1]), (v[1:], v[:-1])):
            assert abs(np.corrcoef(a, b)[0, 1]) < 0.0625


def test_held_roots_follow_the_second_moment():
    """beta2 = 0.999 moves sqrt(v) by under 0.1 % a step, far below half a step of e4m3 (3 to 6 %):
    rounded to nearest it would stay where it began. Dithered, v is right on average: 4096 elements
    whose held v is off by at most about half of itself each (a random walk over steps of a quarter)
    have a mean within 2 % (0.5 / 64 is 0.8 %)."""
    rng = np.random.default_rng(3)
    size, n = np.exp(rng.normal(size=4096)) * 1e-3, 4096
    u, ref, step = np.zeros(n), np.zeros(n), 0
    for phase in (1.0, 2.0):
        gg = (size * np.where(np.arange(n) % 2 == 0, phase, 1.0)) ** 2
        for _ in range(1500):
            step += 1
            r = np.sqrt(0.999 * u * u + 0.001 * gg)
            scale = np.repeat(O.block_scale(r), O.BLOCK)
            u = O.held(r / scale, O.dither(n, step)[1], True) * scale
            ref = 0.999 * ref + 0.001 * gg
        assert abs((u * u / ref).mean() - 1) < 0.02
