"""Plain fp64 oracle (numpy) of the training-step calls around the layer: token embedding and
its gradient, the policy loss and its gradient, AdamW with fp32 and 8-bit states. Test
infrastructure; imports nothing from the product.
"""
import numpy as np

BLOCK = 256


def embed(ids, W, scale):
    y = np.zeros((len(ids), W.shape[1]))
    for t, v in enumerate(ids):
        if 0 <= v < W.shape[0]:
            y[t] = scale * W[v]
    return y


def embed_backward(ids, dy, V, scale, pad=-1, dW0=None):
    """(dW, sum of |terms| per element, terms per row)."""
    dW = np.zeros((V, dy.shape[1])) if dW0 is None else dW0.astype(np.float64).copy()
    mag = np.abs(dW)
    n = np.zeros(V, dtype=np.int64)
    keep = (ids >= 0) & (ids < V) & (ids != pad)
    np.add.at(dW, ids[keep], scale * dy[keep])
    np.add.at(mag, ids[keep], abs(scale) * np.abs(dy[keep]))
    np.add.at(n, ids[keep], 1)
    return dW, mag, n


def log_softmax_at(z, target, tau):
    z = z / tau
    m = z.max(axis=1)
    with np.errstate(invalid="ignore", divide="ignore"):
        lse = m + np.log(np.exp(z - m[:, None]).sum(axis=1))
    return z[np.arange(len(z)), target] - lse


def policy(z, target, adv, old=None, ref=None, w=None, tau=1.0, lo=0.2, hi=0.2, kl=0.0):
    """dict(logp, loss, tok, dz, kept, ratio, size): size bounds |d loss / d logp| term by term."""
    T, V = z.shape
    w = np.ones(T) if w is None else w
    kept = (w != 0) & (target >= 0) & (target < V)
    logp, tok, dz = np.zeros(T), np.zeros(T), np.zeros((T, V))
    ratio, size = np.ones(T), np.zeros(T)
    for t in np.flatnonzero(kept):
        lp = log_softmax_at(z[t:t + 1], target[t:t + 1], tau)[0]
        r = 1.0 if old is None else np.exp(lp - old[t])
        a = adv[t]
        c = np.clip(r, 1 - lo, 1 + hi)
        loss = -min(r * a, c * a)
        slope = -a * r if r * a <= c * a else 0.0
        size[t] = abs(a) * r
        if kl:
            u = ref[t] - lp
            loss += kl * (np.expm1(u) - u)
            slope += kl * (1 - np.exp(u))
            size[t] += abs(kl) * (1 + np.exp(u))
        x = z[t] / tau
        e = np.exp(x - x.max())
        p = e / e.sum()
        g = -p
        g[target[t]] += 1
        logp[t], tok[t], dz[t], ratio[t] = lp, w[t] * loss, w[t] * slope / tau * g, r
    return dict(logp=logp, loss=tok.sum(), tok=tok, dz=dz, kept=kept, ratio=ratio, size=size)


def adamw(x, g, m, v, step, lr, b1, b2, eps, decay):
    """One step (the step-th, from 1): new x, m, v and the update's size."""
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    up = lr * (m / (1 - b1 ** step)) / (np.sqrt(v / (1 - b2 ** step)) + eps)
    return x * (1 - lr * decay) - up, m, v, np.abs(up)


# ---------------------------------------------------------------- 8-bit states

def e4m3_values():
    """Value of each of the 256 codes (sign, 4 exponent bits with bias 7, 3 mantissa bits; no
    infinities, 0x7f and 0xff are NaN)."""
    out = np.empty(256)
    for c in range(256):
        s, e, f = -1.0 if c & 0x80 else 1.0, (c >> 3) & 15, c & 7
        out[c] = s * (f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
    out[0x7f] = out[0xff] = np.nan
    return out


def dither(n, step, start=0):
    """20 bits for each element and step, twice: for m and for v."""
    i = np.arange(start, start + n, dtype=np.uint64)
    low, c, e = np.uint64(0xFFFFFFFF), np.uint64(0x85EBCA6B), np.uint64(0xC2B2AE35)
    with np.errstate(over="ignore"):
        h = (i * np.uint64(0x9E3779B1) + np.uint64(step * 0x61C88647)) & low
        h = ((h ^ (h >> np.uint64(15))) * c) & low
        return (h >> np.uint64(12)).astype(np.float64), (((h * e) & low) >> np.uint64(12)).astype(np.float64)


def weyl(n, step, start=0):
    """The 20 bits of a Weyl sequence over elements and steps, for m; for v with the top bit turned."""
    i = np.arange(start, start + n, dtype=np.uint64)
    with np.errstate(over="ignore"):
        d = ((i * np.uint64(0x9E3779B1) + np.uint64(step * 0x61C88647)) & np.uint64(0xFFFFFFFF)) >> np.uint64(12)
    return d.astype(np.float64), (d ^ np.uint64(0x80000)).astype(np.float64)


def blocks(x):
    n = len(x)
    return np.pad(x, (0, -n % BLOCK)).reshape(-1, BLOCK)


def block_scale(x):
    """The power of two that leaves the largest finite magnitude of each block in [128, 256)."""
    top = np.where(np.isfinite(blocks(x)), np.abs(blocks(x)), 0.0).max(axis=1)
    return np.where(top > 0, 2.0 ** (np.floor(np.log2(np.where(top > 0, top, 1.0))) - 7), 0.0)


def held(y, d, root, even=True):
    """The e4m3 value that y is held as: one of its two neighbours on the grid, the upper one where
    the share of the way to it, of y or (a root, evened in its square) of y^2, and the dither d (20
    bits) come to 1. A root above zero keeps the least step."""
    a = np.abs(y)
    unit = 2.0 ** np.maximum(np.floor(np.log2(np.where(a > 0, a, 1e-30))) - 3, -9)
    low = np.floor(a / unit) * unit
    k = 2 if root and even else 1
    share = (a ** k - low ** k) / ((low + unit) ** k - low ** k)
    q = np.where(share + d / 2 ** 20 >= 1, low + unit, low)
    if root:
        q = np.where(a > 0, np.maximum(q, 2.0 ** -9), q)
    return np.sign(y) * q
