"""The rounding rules of 8-bit AdamW states on the CPU: the Weyl rule of the oracle against the
rule's own words and a form written apart from it, and refusals."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import train_oracle as O


def test_weyl_words():
    for i, step in ((0, 1), (1, 1), (77, 21), (2 ** 32 + 77, 21), (2 ** 33 - 1, 10 ** 6)):
        d = (i * 0x9E3779B1 + step * 0x61C88647) % 2 ** 32 // 2 ** 12
        m, v = O.weyl(1, step, start=i)
        assert m[0] == d and v[0] == (d + 2 ** 19) % 2 ** 20      # v's top bit is turned


def test_weyl_words_cover_steps_evenly():
    """Over any run of steps the dither of one element is spread like a golden-ratio sequence: the words'
    factor of the step is 2^32 over the golden ratio's square."""
    for i in (0, 5, 12345):
        for k in (0, 1):
            d = np.sort([O.weyl(1, s, start=i)[k][0] for s in range(1, 257)]) / 2 ** 20
            assert np.diff(d).max() < 3 / 256 and d[0] < 3 / 256 and d[-1] > 1 - 3 / 256


@pytest.mark.parametrize("root", [False, True])
def test_weyl_rounding(root):
    """Down to the grid after the dither's part of a grid step was added; exact on grid values; right on
    average over the dither in the value itself; a root above zero keeps the least step."""
    grid = np.sort(O.e4m3_values()[:121])
    rng = np.random.default_rng(2)
    y = np.concatenate([rng.uniform(0, 255, 500), rng.uniform(0, 2.0 ** -5, 500), grid]).astype(np.float32)
    d = rng.integers(0, 1 << 20, len(y))
    # the rule on the bits of fp32 numbers, and on multiples of 2^-9 below 2^-6
    bits = ((y.view(np.int32).astype(np.int64) + d) & ~0xFFFFF).astype(np.int32).view(np.float32)
    want = np.where(y < 2.0 ** -6, np.floor(y.astype(np.float64) * 512 + d / 2 ** 20) / 512, bits)
    if root:
        want = np.where((y > 0) & (want == 0), 2.0 ** -9, want)
    got = O.held(y.astype(np.float64), d.astype(float), root, even=False)
    assert np.array_equal(got, want) and np.isin(got, grid).all() and (got[-len(grid):] == grid).all()
    every = np.arange(0, 1 << 20, 64, dtype=float)
    for a in ((0.0057,) if root else (0.0007, 0.0057)) + (0.013, 1.03, 77.7, 231.0):
        unit = 2.0 ** max(np.floor(np.log2(a)) - 3, -9)
        assert abs(O.held(np.full(len(every), a), every, root, even=False).mean() - a) < unit * 64 / 2 ** 20
    assert O.held(np.array([1e-9, 0.0]), np.zeros(2), True, even=False).tolist() == [2.0 ** -9, 0.0]


def test_refusals(moe_lib):
    """A rounding that is none, and a reserved field that is set, before anything is launched."""
    lib, p = moe_lib.load(), ctypes.c_void_p(256)
    t = (moe_lib._lib.MoeAdamwTensor * 1)()
    t[0].p = t[0].g = t[0].m = t[0].v = 256
    t[0].n, t[0].dtype = 100, 1
    for bad in (dict(rounding=2), dict(rounding=-1), dict(reserved=1)):
        c = moe_lib._lib.MoeAdamwConfig(1e-3, 0.9, 0.999, 1e-8)
        for k, v in bad.items():
            setattr(c, k, v)
        assert lib.moe_adamw(ctypes.byref(c), t, 1, None, None, p, None) == moe_lib.MOE_ERR_INVALID_ARG
    x = torch.zeros(300)
    with pytest.raises(ValueError):
        moe_lib.AdamW([dict(p=x, g=x.clone())], bits=8, rounding="nearest")
    assert moe_lib.AdamW([dict(p=x, g=x.clone())], bits=8).cfg.rounding == 0
    assert moe_lib.AdamW([dict(p=x, g=x.clone())], bits=8, rounding="weyl").cfg.rounding == 1
