"""Refusals of scored routing, layer norm and Muon, on the host: a bad configuration, a missing or
misaligned array is refused before any launch (the addresses here are not real)."""
import ctypes

import pytest
import torch

P, Q = ctypes.c_void_p(256), ctypes.c_void_p(258)
R = ctypes.c_void_p(512)
BAD, NOT = -1, -2


def ref(c):
    return ctypes.byref(c)


def put(c, /, **kw):
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def scores_cfg(moe, **kw):
    return put(moe.make_score_config(10, 16, 4, groups=4, groups_kept=2), **kw)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), BAD), (dict(E=0), BAD), (dict(E=257), BAD), (dict(k=0), BAD), (dict(k=9), BAD), (dict(groups=3), BAD),
    (dict(groups=0), BAD), (dict(groups_kept=0), BAD), (dict(groups_kept=5), BAD), (dict(groups_kept=1, k=5), BAD),
    (dict(E=256, groups=64), BAD), (dict(group_top=3), BAD), (dict(group_top=0), BAD), (dict(score=2), BAD),
    (dict(renormalise=2), BAD), (dict(temperature=0.0), BAD), (dict(temperature=float("inf")), BAD),
    (dict(temperature=float("nan")), BAD), (dict(temperature=1e-39), BAD), (dict(scale=float("nan")), BAD),
    (dict(T=2 ** 27 + 1), NOT)])
def test_scores_refuse_configs(moe_lib, bad, status):
    lib, c = moe_lib.load(), scores_cfg(moe_lib, **bad)
    assert lib.moe_route_scores(ref(c), P, P, P, P, P, P, P, None) == status
    assert lib.moe_route_scores_backward(ref(c), P, P, P, P, None) == status
    assert lib.moe_route_scores_workspace_bytes(ref(c)) == 0


def test_scores_refuse_arrays(moe_lib):
    lib, c = moe_lib.load(), scores_cfg(moe_lib)
    for i in range(7):
        for p in (None, Q):
            if p is None and i in (1, 4, 5):            # bias, counts and balance_loss may be missing
                continue
            if p is Q and i not in (0, 6):              # 4-byte arrays: an odd address instead
                p = ctypes.c_void_p(257)
            args = [P] * 7
            args[i] = p
            assert lib.moe_route_scores(ref(c), *args, None) == BAD
    for i in range(4):
        for p in (None, ctypes.c_void_p(257)):
            args = [P, P, P, R]
            args[i] = p
            assert lib.moe_route_scores_backward(ref(c), *args, None) == BAD
    assert lib.moe_route_scores_backward(ref(c), P, P, P, P, None) == BAD       # dlogits in place of logits
    assert lib.moe_route_scores(None, P, P, P, P, P, P, P, None) == BAD
    c = scores_cfg(moe_lib, T=0)
    assert lib.moe_route_scores(ref(c), None, None, None, None, None, None, None, None) == 0
    assert lib.moe_route_scores_backward(ref(c), None, None, None, None, None) == 0


def test_backward_scores_refuses(moe_lib):
    moe, lib = moe_lib, moe_lib.load()
    c = moe.make_config(10, 64, 16, 4, 64)
    good = [P, R] + [P] * 25 + [None]

    def call(c, s, args=good):
        return lib.moe_backward_scores(ref(c), s if s is None else ref(s), *args)
    assert call(c, None) == BAD
    for bad in (dict(T=9), dict(E=8), dict(k=3), dict(score=9)):
        assert call(c, scores_cfg(moe, **bad)) == BAD
    for i in (0, 1):                                    # logits, dlogits
        for p in (None, Q):
            args = list(good)
            args[i] = p
            assert call(c, scores_cfg(moe), args) == BAD
    assert call(c, scores_cfg(moe), [P] * 27 + [None]) == BAD                   # dlogits in place of logits
    dense = moe.make_config(10, 64, 4, 4, 64)
    assert call(dense, put(moe.make_score_config(10, 4, 4))) == NOT


def norm_cfg(moe, **kw):
    return put(moe.make_norm_config(10, 64), **kw)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), BAD), (dict(d=0), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(dtype=2), BAD),
    (dict(param_dtype=-1), BAD), (dict(accumulate=2), BAD), (dict(T=2 ** 30 + 1), NOT), (dict(d=2 ** 20 + 1), NOT)])
def test_norm_refuses_configs(moe_lib, bad, status):
    lib, c = moe_lib.load(), norm_cfg(moe_lib, **bad)
    assert lib.moe_layer_norm(ref(c), P, None, P, P, None, P, P, P, None) == status
    assert lib.moe_layer_norm_backward(ref(c), P, P, P, P, P, P, P, P, R, P, None) == status
    assert lib.moe_norm_workspace_bytes(ref(c)) == 0


def test_norm_refuses_arrays(moe_lib):
    lib, c = moe_lib.load(), norm_cfg(moe_lib)
    good = [P, P, P, P, R, P, P, P]                     # x, residual, gain, bias, total, y, mean, rstd
    for i in range(6):
        args = list(good)
        args[i] = Q
        assert lib.moe_layer_norm(ref(c), *args, None) == BAD
    for i in (0, 1, 4, 5):                              # residual and total: both or neither
        args = list(good)
        args[i] = None
        assert lib.moe_layer_norm(ref(c), *args, None) == BAD
    assert lib.moe_layer_norm(ref(c), P, P, P, P, R, R, P, P, None) == BAD      # y is total
    good = [P, P, P, P, P, P, P, P, R, P]               # dy, s, gain, mean, rstd, dtotal, dx, dgain, dbias, ws
    for i in range(10):
        args = list(good)
        args[i] = ctypes.c_void_p(257)
        assert lib.moe_layer_norm_backward(ref(c), *args, None) == BAD
    for i in (0, 1, 3, 4, 9):
        args = list(good)
        args[i] = None
        assert lib.moe_layer_norm_backward(ref(c), *args, None) == BAD
    assert lib.moe_layer_norm_backward(ref(c), P, P, P, P, P, P, None, None, None, P, None) == BAD   # nothing wanted
    assert lib.moe_layer_norm_backward(ref(c), P, P, P, P, P, P, P, R, R, P, None) == BAD            # one array twice
    c = norm_cfg(moe_lib, T=0)
    assert lib.moe_layer_norm(ref(c), None, None, None, None, None, None, None, None, None) == 0
    c.accumulate = 1
    assert lib.moe_layer_norm_backward(ref(c), None, None, None, None, None, None, None, P, R, P, None) == 0


def muon_cfg(moe, **kw):
    return put(moe.make_muon_config(2, 64, 32), **kw)


@pytest.mark.parametrize("bad,status", [
    (dict(count=-1), BAD), (dict(rows=0), BAD), (dict(cols=0), BAD), (dict(steps=-1), BAD), (dict(steps=101), BAD),
    (dict(a=17.0), BAD), (dict(b=float("nan")), BAD), (dict(c=-16.5), BAD), (dict(lr=float("inf")), BAD),
    (dict(lr=1e39), BAD), (dict(momentum=1.0), BAD), (dict(momentum=-0.1), BAD), (dict(weight_decay=float("nan")), BAD),
    (dict(scale=float("inf")), BAD), (dict(eps=0.0), BAD), (dict(eps=2.0), BAD), (dict(nesterov=2), BAD),
    (dict(dtype=2), BAD), (dict(grad_dtype=-1), BAD), (dict(precision=5), BAD), (dict(count=65536), NOT),
    (dict(rows=65537), NOT), (dict(cols=65537), NOT), (dict(count=65535, rows=65536, cols=65536), NOT)])
def test_muon_refuses_configs(moe_lib, bad, status):
    lib, c = moe_lib.load(), muon_cfg(moe_lib, **bad)
    assert lib.moe_orthogonalize(ref(c), P, P, P, None) == status
    assert lib.moe_muon(ref(c), P, P, P, P, P, P, P, None) == status
    assert lib.moe_muon_workspace_bytes(ref(c)) == 0


def test_muon_refuses_arrays(moe_lib):
    lib, c = moe_lib.load(), muon_cfg(moe_lib)
    for i in range(3):
        for p in (None, Q):
            args = [P, P, P]
            args[i] = p
            assert lib.moe_orthogonalize(ref(c), *args, None) == BAD
    for i in range(7):
        args = [P] * 7
        args[i] = ctypes.c_void_p(257)
        assert lib.moe_muon(ref(c), *args, None) == BAD
        if i in (0, 1, 3, 6):                           # master, lr and grad_scale may be missing
            args[i] = None
            assert lib.moe_muon(ref(c), *args, None) == BAD
    assert 0 < moe_lib.muon_workspace_bytes(moe_lib.make_muon_config(1000, 128, 1024)) < 4096
    assert moe_lib.muon_workspace_bytes(moe_lib.make_muon_config(2, 129, 1024)) > 4 * 129 * 1024 * 2
    c.grad_dtype = moe_lib.MOE_F32
    assert lib.moe_orthogonalize(ref(c), P, P, R, None) == BAD      # in place, but of another type
    c.count = 0
    assert lib.moe_orthogonalize(ref(c), None, None, None, None) == 0
    assert lib.moe_muon(ref(c), None, None, None, None, None, None, None, None) == 0


F, I, B = torch.float32, torch.int32, torch.bfloat16


def z(*shape, dtype=F):
    return torch.zeros(*shape, dtype=dtype)


def test_host_tensors_are_refused(moe_lib):
    moe = moe_lib
    c = moe.make_score_config(4, 8, 2)
    with pytest.raises(ValueError, match="GPU"):
        moe.route_scores(c, z(4, 8), None, z(4, 2, dtype=I), z(4, 2))
    with pytest.raises(ValueError, match="GPU"):
        moe.route_scores_backward(c, z(4, 8), z(4, 2, dtype=I), z(4, 2), z(4, 8))
    c = moe.make_norm_config(4, 8)
    x = z(4, 8, dtype=B)
    with pytest.raises(ValueError, match="GPU"):
        moe.layer_norm(c, x, z(8), z(8), x)
    with pytest.raises(ValueError, match="GPU"):
        moe.layer_norm_backward(c, x, x, z(8), z(4), z(4), x, None, None, None)
    c = moe.make_muon_config(2, 8, 4)
    ws = z(moe.muon_workspace_bytes(c), dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        moe.orthogonalize(c, z(2, 8, 4, dtype=B), z(2, 8, 4, dtype=B), ws)
    opt = moe.Muon([dict(p=z(2, 8, 4), g=z(2, 8, 4)), dict(p=z(8, 4, dtype=B), g=z(8, 4, dtype=B), master=z(8, 4))])
    with pytest.raises(ValueError, match="GPU"):
        opt.step()
    moe.Muon([]).step()
    moe.Muon([dict(p=z(0, 8, 4), g=z(0, 8, 4))]).step()


def test_binding_refuses_wrong_arrays(moe_lib):
    moe = moe_lib
    c = moe.make_score_config(4, 8, 2)
    for bad in (dict(logits=z(4, 7)), dict(logits=z(4, 8, dtype=B)), dict(logits=z(4, 16)[:, ::2]), dict(bias=z(7)),
                dict(idx=z(4, 2)), dict(w=z(4, 3)), dict(counts=z(8)), dict(balance_loss=z(2))):
        a = dict(logits=z(4, 8), bias=None, idx=z(4, 2, dtype=I), w=z(4, 2))
        a.update(bad)
        with pytest.raises(ValueError):
            moe.route_scores(c, **a, ws=z(4096))
    with pytest.raises(ValueError, match="ws"):
        moe.route_scores(c, z(4, 8), None, z(4, 2, dtype=I), z(4, 2), counts=z(8, dtype=I))
    with pytest.raises(ValueError, match="score"):
        moe.make_score_config(4, 8, 2, score="relu")
    c = moe.make_norm_config(4, 8)
    x = z(4, 8, dtype=B)
    with pytest.raises(ValueError, match="total"):
        moe.layer_norm(c, x, None, None, x, residual=x)
    with pytest.raises(ValueError, match="residual"):
        moe.layer_norm(c, x, None, None, x, total=x)
    with pytest.raises(ValueError, match="gain"):
        moe.layer_norm(c, x, z(8, dtype=B), None, x)
    with pytest.raises(ValueError, match="ws"):
        moe.layer_norm_backward(c, x, x, None, z(4), z(4), x, z(8), None, None)
    with pytest.raises(ValueError, match="dtotal"):
        moe.layer_norm_backward(c, x, x, None, z(4), z(4), x, None, None, None, dtotal=z(4, 8))
    p = z(8, 4)
    for bad in (dict(p=z(8), g=z(8)), dict(p=p, g=z(4, 8)), dict(p=p, g=p.half()), dict(p=p, g=z(4, 8).t()),
                dict(p=p, g=p, m=z(8, 4, dtype=B)), dict(p=p, g=p, master=z(4, 8))):
        with pytest.raises(ValueError):
            moe.Muon([bad])
    with pytest.raises(moe.MoeError):
        moe.Muon([dict(p=p, g=p)], momentum=1.5)
