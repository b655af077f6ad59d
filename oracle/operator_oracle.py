"""Plain fp64 oracle (numpy) of layer norm, the choice of experts from scores and orthogonalised
updates (Muon), with their gradients. Test infrastructure; imports nothing from the product.
"""
import numpy as np

TINY = 1e-20      # added to the sum of the chosen sigmoids


# ---------------------------------------------------------------- choice of experts

def scores(z, kind, tau):
    x = z / tau
    with np.errstate(invalid="ignore", over="ignore"):
        if kind == "sigmoid":
            return 1 / (1 + np.exp(-x))
        m = x.max(axis=1, keepdims=True)
        e = np.exp(x - np.where(np.isneginf(m), 0, m))
        t = e.sum(axis=1, keepdims=True)
        p = np.where(t > 0, e / np.where(t > 0, t, 1), 0)
        bad = np.isnan(x).any(axis=1) | np.isposinf(x).any(axis=1)
        p[bad] = np.nan
        return p


def choose(z, bias, kind, k, groups=1, kept=1, top=1, tau=1.0):
    """(idx [T, k], score [T, E], gap [T]): gap is the smallest distance between two values of which
    one was taken before the other (experts in the choice's order, the border included; groups at
    theirs). Ties go to the lower id."""
    T, E = z.shape
    s = scores(z, kind, tau)
    by_logit = bias is None and (kept == groups or top == 1)
    c = z.astype(np.float64).copy() if by_logit else s + (0 if bias is None else bias)
    with np.errstate(invalid="ignore"):
        c[np.isnan(c) | np.isneginf(z)] = -np.inf
    if kind == "softmax":
        c[np.isnan(s).any(axis=1)] = -np.inf
    idx, gap = np.zeros((T, k), dtype=np.int64), np.full(T, np.inf)
    size = E // groups
    for t in range(T):
        v = c[t].copy()
        if kept < groups:
            rows = -np.sort(-v.reshape(groups, size), axis=1)
            worth = rows[:, 0] + (rows[:, 1] if top == 2 and size > 1 else 0)
            worth[np.isnan(worth)] = -np.inf
            order = np.argsort(-worth, kind="stable")
            if np.isfinite(worth[order[kept]]):
                gap[t] = worth[order[kept - 1]] - worth[order[kept]]
            shut = np.ones(groups, dtype=bool)
            shut[order[:kept]] = False
            v[np.repeat(shut, size)] = np.nan          # below everything, -inf included
        order = np.argsort(np.where(np.isnan(v), np.inf, -v), kind="stable")
        order = np.concatenate([order[~np.isnan(v[order])], order[np.isnan(v[order])]])
        idx[t] = order[:k]
        w = v[order[:k + 1]]
        for a, b in zip(w[:-1], w[1:]):
            if np.isfinite(a) and np.isfinite(b):
                gap[t] = min(gap[t], a - b)
    return idx, s, gap


def weights(z, s, idx, kind, renorm, scale, tau):
    w = np.take_along_axis(s, idx, axis=1)
    if renorm and kind == "softmax":
        bad = np.isnan(s).any(axis=1)
        w = scores(np.take_along_axis(z, idx, axis=1).astype(np.float64), "softmax", tau)
        w[bad] = np.nan
    elif renorm:
        w = w / (w.sum(axis=1, keepdims=True) + TINY)
    return scale * w


def counts(idx, E):
    n = np.bincount(idx.reshape(-1), minlength=E)
    return n, np.mean((n - idx.size / E) ** 2)


def scores_backward(z, idx, dw, kind, renorm, scale, tau):
    """(dz, size): size bounds dz term by term."""
    T, E = z.shape
    s = scores(z, kind, tau)
    dz, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        i = idx[t]
        if kind == "softmax" and renorm:
            share = scores(z[t:t + 1, i].astype(np.float64), "softmax", tau)[0]
            diff = dw[t][:, None] - dw[t][None, :]
            dz[t, i] = scale * share * (diff * share[None, :]).sum(1) / tau
            size[t, i] = scale * share * (np.abs(diff) * share[None, :]).sum(1) / tau
            continue
        p = s[t, i]
        if renorm:
            tot = p.sum() + TINY
            diff = dw[t][:, None] - dw[t][None, :]
            g = scale / tot * ((diff * (p / tot)[None, :]).sum(1) + dw[t] * TINY / tot)
            a = scale / tot * ((np.abs(diff) * (p / tot)[None, :]).sum(1) + np.abs(dw[t]) * TINY / tot)
        else:
            g, a = scale * dw[t], abs(scale) * np.abs(dw[t])
        if kind == "sigmoid":
            with np.errstate(over="ignore"):
                slope = p / (1 + np.exp(z[t, i] / tau))
            dz[t, i], size[t, i] = g * slope / tau, a * slope / tau
        else:
            full, fa = np.zeros(E), np.zeros(E)
            full[i], fa[i] = g, a
            dz[t] = s[t] * (full - (p * g).sum()) / tau
            size[t] = s[t] * (fa + (p * a).sum()) / tau
    return dz, size


# ---------------------------------------------------------------- layer norm

def norm(x, gain, bias, eps):
    mean = x.mean(axis=1)
    h = x - mean[:, None]
    rstd = 1 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * gain + bias, mean, rstd


def norm_backward(dy, x, gain, mean, rstd):
    h = (x - mean[:, None]) * rstd[:, None]
    g = dy * gain
    dx = rstd[:, None] * (g - g.mean(axis=1, keepdims=True) - h * (g * h).mean(axis=1, keepdims=True))
    return dx, (dy * h).sum(axis=0), dy.sum(axis=0)


# ---------------------------------------------------------------- orthogonalised updates

def orth(u, steps=5, coef=(3.4445, -4.7750, 2.0315), eps=1e-7, held=None):
    """Newton-Schulz steps on one matrix. `held(x, what)` is what storage makes of an operand ("X", "A",
    "B" without its diagonal); `held(x, ("sum", K))` of a product of length K. (With held = fp16_planes(1)
    X is rounded to one fp16 number, which the kernels do not; orth_one_part has their roundings.)"""
    a, b, c = coef
    keep = held or (lambda x, what: x)
    tall = u.shape[0] > u.shape[1]
    x = keep(u / (np.sqrt((u * u).sum()) + eps), "X")
    eye = np.eye(min(u.shape))
    for _ in range(steps):
        A = keep(keep(x.T @ x if tall else x @ x.T, ("sum", max(u.shape))), "A")
        B = a * eye + b * A + c * keep(A @ A, ("sum", min(u.shape)))
        D = np.diag(np.diag(B))
        B = keep(B - D, "B")
        x = keep(keep(x @ B if tall else B @ x, ("sum", min(u.shape))) + (x @ D if tall else D @ x), "X")
    return x


def fp16_planes(planes):
    """Storage as the kernels have it: X and A times 2^11, B times 2^10, in one fp16 number or two; with
    two, sums lose up to 2^-23 of themselves with each of K / 16 additions to each of three terms."""
    scale = {"X": 2.0 ** 11, "A": 2.0 ** 11, "B": 2.0 ** 10}

    def held(x, what):
        if isinstance(what, tuple):
            return x if planes == 1 else x * (1 - 2.0 ** -23 * 3 * np.ceil(what[1] / 16))
        y = x * scale[what]
        hi = y.astype(np.float16).astype(np.float64)
        return (hi if planes == 1 else hi + (y - hi).astype(np.float16).astype(np.float64)) / scale[what]
    return held


def two_parts(adds=24, seed=0):
    """Storage in two fp16 parts, as fp16_planes(2), and sums as the tensor cores leave them where at most `adds`
    additions go to one partial sum: each cuts off up to 2^-24 of it (more or less in one element than in the next:
    what the cuts have in common shrinks a product, what differs stands in all directions)."""
    held, rng = fp16_planes(2), np.random.default_rng(seed)
    return lambda x, what: x * (1 - 2.0 ** -24 * adds * rng.random(x.shape)) if isinstance(what, tuple) else held(x, what)


def orth_one_part(u, steps=5, coef=(3.4445, -4.7750, 2.0315), eps=1e-7):
    """orth as the kernels round it with one-part products: A and B without its diagonal in one fp16 number; X in
    two, of which the Gram product takes the high one, the last product both but for the last two steps, and
    the diagonal of B both."""
    a, b, c = coef
    one, two = fp16_planes(1), fp16_planes(2)
    tall = u.shape[0] > u.shape[1]
    x = two(u / (np.sqrt((u * u).sum()) + eps), "X")
    eye = np.eye(min(u.shape))
    for k in range(steps):
        hi = one(x, "X")
        A = one(hi.T @ hi if tall else hi @ hi.T, "A")
        B = a * eye + b * A + c * (A @ A)
        D = np.diag(np.diag(B))
        B = one(B - D, "B")
        y = x if k + 2 < steps else hi
        x = two((y @ B if tall else B @ y) + (x @ D if tall else D @ x), "X")
    return x


def muon(p, g, m, lr, momentum, decay, scale, nesterov, **kw):
    m = momentum * m + g
    u = g + momentum * m if nesterov else m
    return p * (1 - lr * decay) - lr * scale * orth(u, **kw), m
