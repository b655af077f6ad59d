"""Gradients of the fp64 oracle of norm and scored routing, against differences; its orthogonalisation
against the polynomial on singular values."""
import numpy as np
import pytest

from oracle import operator_oracle as O


def differences(f, x, h):
    """Central differences of the scalar f, whose error is h^2 times the third derivative."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("tau", [1.0, 0.5])
def test_scores_gradient(kind, renorm, tau):
    r = np.random.default_rng(0)
    z, dw = r.normal(size=(4, 9)), r.normal(size=(4, 3))
    idx, _, _ = O.choose(z, None, kind, 3, tau=tau)
    dz, size = O.scores_backward(z, idx, dw, kind, renorm, 2.5, tau)

    def f(v):
        return (O.weights(v, O.scores(v, kind, tau), idx, kind, renorm, 2.5, tau) * dw).sum()
    # h = 1e-5: h^2 times third derivatives of order 2.5 / tau^3, and 1e-16 / h of rounding
    assert np.abs(dz - differences(f, z, 1e-5)).max() < 1e-8
    assert (np.abs(dz) <= size * (1 + 1e-12)).all()


def test_norm_gradient():
    r = np.random.default_rng(1)
    x, gain, bias, dy = r.normal(size=(3, 7)), r.normal(size=7), r.normal(size=7), r.normal(size=(3, 7))
    _, mean, rstd = O.norm(x, gain, bias, 1e-5)
    dx, dgain, dbias = O.norm_backward(dy, x, gain, mean, rstd)
    assert np.abs(dx - differences(lambda v: (O.norm(v, gain, bias, 1e-5)[0] * dy).sum(), x, 1e-5)).max() < 1e-7
    assert np.abs(dgain - differences(lambda v: (O.norm(x, v, bias, 1e-5)[0] * dy).sum(), gain, 1e-5)).max() < 1e-8
    assert np.abs(dbias - differences(lambda v: (O.norm(x, gain, v, 1e-5)[0] * dy).sum(), bias, 1e-5)).max() < 1e-8


@pytest.mark.parametrize("shape", [(5, 5), (4, 9), (9, 4), (1, 6), (6, 1)])
def test_orth_is_a_polynomial_of_the_singular_values(shape):
    u = np.random.default_rng(2).normal(size=shape)
    left, s, right = np.linalg.svd(u, full_matrices=False)
    s = s / (np.sqrt((s * s).sum()) + 1e-7)
    for _ in range(5):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    assert np.abs(O.orth(u) - (left * s) @ right).max() < 1e-12
    assert (O.orth(np.zeros(shape)) == 0).all()


def test_choice_by_hand():
    z = np.array([[0.0, 2.0, 2.0, 1.0], [-np.inf, -np.inf, -np.inf, 3.0], [np.nan, 1.0, 2.0, 3.0]])
    idx, _, _ = O.choose(z, None, "sigmoid", 2)
    assert idx.tolist() == [[1, 2], [3, 0], [3, 2]]
    idx, _, _ = O.choose(z, None, "softmax", 2)
    assert idx.tolist() == [[1, 2], [3, 0], [0, 1]]            # a row with NaN has no softmax
    idx, _, _ = O.choose(z[:1], None, "sigmoid", 2, groups=2, kept=1)
    assert idx.tolist() == [[1, 0]]                            # groups tie at 2: the first
    idx, _, _ = O.choose(z[:1], None, "sigmoid", 2, groups=2, kept=1, top=2)
    assert idx.tolist() == [[2, 3]]
    idx, _, _ = O.choose(z[:1], np.array([0, -1.0, 0, 0]), "sigmoid", 2)
    assert idx.tolist() == [[2, 3]]
