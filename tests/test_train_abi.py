"""Refusals of the training-step calls, on the host: a bad configuration, a missing or
misaligned array is refused before any launch (the addresses here are not real)."""
import ctypes

import pytest
import torch

P, Q = ctypes.c_void_p(256), ctypes.c_void_p(258)


def embed_cfg(moe, **kw):
    c = moe.make_embed_config(10, 20, 8)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), -1), (dict(V=0), -1), (dict(d=0), -1), (dict(scale=float("nan")), -1), (dict(padding_id=20), -1),
    (dict(padding_id=-2), -1), (dict(dtype=5), -1), (dict(grad_dtype=-1), -1), (dict(accumulate=2), -1),
    (dict(T=2 ** 31 - 1), -2), (dict(V=2 ** 31 - 1), -2), (dict(d=2 ** 31 - 1), -2)])
def test_embed_refuses_configs(moe_lib, bad, status):
    lib, c = moe_lib.load(), embed_cfg(moe_lib, **bad)
    assert lib.moe_embed(ctypes.byref(c), P, P, P, None) == status
    assert lib.moe_embed_backward(ctypes.byref(c), P, P, P, P, None) == status
    assert lib.moe_embed_workspace_bytes(ctypes.byref(c)) == 0


@pytest.mark.parametrize("i", range(3))
@pytest.mark.parametrize("p", [None, Q])
def test_embed_refuses_arrays(moe_lib, i, p):
    lib, c, args = moe_lib.load(), embed_cfg(moe_lib), [P] * 3
    args[i] = p
    assert lib.moe_embed(ctypes.byref(c), *args, None) == moe_lib.MOE_ERR_INVALID_ARG
    for j in range(4):
        args = [P] * 4
        args[j] = p
        assert lib.moe_embed_backward(ctypes.byref(c), *args, None) == moe_lib.MOE_ERR_INVALID_ARG
    assert lib.moe_embed(None, P, P, P, None) == moe_lib.MOE_ERR_INVALID_ARG


def test_embed_nothing_to_do(moe_lib):
    c = embed_cfg(moe_lib, T=0)
    assert moe_lib.load().moe_embed(ctypes.byref(c), None, P, None, None) == 0
    assert moe_lib.embed_workspace_bytes(c) > 0


def policy_cfg(moe, **kw):
    c = moe.make_policy_config(10, 21, kl_weight=0.1)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), -1), (dict(V=0), -1), (dict(ld=20), -1), (dict(ld_grad=20), -1), (dict(dtype=3), -1),
    (dict(temperature=0.0), -1), (dict(temperature=float("inf")), -1), (dict(temperature=1e-39), -1),
    (dict(clip_low=1.5), -1), (dict(clip_low=-0.1), -1), (dict(clip_high=-0.1), -1),
    (dict(clip_high=float("inf")), -1), (dict(kl_weight=float("nan")), -1),
    (dict(V=2 ** 30 + 1, ld=2 ** 31, ld_grad=2 ** 31), -2), (dict(ld=2 ** 41), -2), (dict(ld_grad=2 ** 41), -2)])
def test_policy_refuses_configs(moe_lib, bad, status):
    lib, c = moe_lib.load(), policy_cfg(moe_lib, **bad)
    assert lib.moe_policy_loss(ctypes.byref(c), *[P] * 10, None) == status
    assert lib.moe_token_logp(ctypes.byref(c), P, P, P, None) == status
    assert lib.moe_policy_workspace_bytes(ctypes.byref(c)) == 0


def test_policy_refuses_arrays(moe_lib):
    lib, c, inval = moe_lib.load(), policy_cfg(moe_lib), moe_lib.MOE_ERR_INVALID_ARG
    Z = ctypes.c_void_p(4096)
    # logits target advantage old ref weight logp loss dlogits ws
    good = [P, P, P, P, P, P, P, P, Z, P]
    for i in range(10):
        args = list(good)
        args[i] = ctypes.c_void_p(257)
        assert lib.moe_policy_loss(ctypes.byref(c), *args, None) == inval
    for i in (0, 1, 2, 4, 9):                  # ref_logp is needed for the KL term, ws for the loss
        args = list(good)
        args[i] = None
        assert lib.moe_policy_loss(ctypes.byref(c), *args, None) == inval
    c2 = policy_cfg(moe_lib, ld=32)            # in place needs one stride
    assert lib.moe_policy_loss(ctypes.byref(c2), P, P, P, P, P, P, P, P, P, P, None) == inval
    for i in range(3):
        for p in (None, ctypes.c_void_p(257)):
            args = [P] * 3
            args[i] = p
            assert lib.moe_token_logp(ctypes.byref(c), *args, None) == inval


def adam_table(moe, n=1, **kw):
    t = (moe._lib.MoeAdamwTensor * n)()
    for e in t:
        e.p = e.g = e.m = e.v = 256
        e.n, e.dtype, e.grad_dtype = 100, 1, 0
        for k, v in kw.items():
            setattr(e, k, v)
    return t


@pytest.mark.parametrize("bad,status", [
    (dict(n=-1), -1), (dict(reserved=1), -1), (dict(dtype=9), -1), (dict(grad_dtype=2), -1),
    (dict(weight_decay=-0.1), -1), (dict(weight_decay=float("nan")), -1), (dict(m_scale=256), -1),
    (dict(v_scale=256), -1), (dict(p=0), -1), (dict(g=0), -1), (dict(m=0), -1), (dict(v=0), -1), (dict(p=258), -1),
    (dict(g=260), -1), (dict(master=260), -1), (dict(m=260), -1), (dict(v=264), -1),
    (dict(m_scale=258, v_scale=256), -1), (dict(n=2 ** 38 + 1), -2)])
def test_adamw_refuses_tensors(moe_lib, bad, status):
    lib, c = moe_lib.load(), moe_lib._lib.MoeAdamwConfig(1e-3, 0.9, 0.999, 1e-8)
    for n in (1, 3):
        t = adam_table(moe_lib, n)
        for k, v in bad.items():
            setattr(t[n - 1], k, v)
        assert lib.moe_adamw(ctypes.byref(c), t, n, None, None, P, None) == status


@pytest.mark.parametrize("bad", [dict(lr=float("inf")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
                                 dict(beta2=float("nan")), dict(eps=0.0), dict(eps=1e-31), dict(eps=float("inf"))])
def test_adamw_refuses_settings(moe_lib, bad):
    lib, kw = moe_lib.load(), dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8)
    kw.update(bad)
    c = moe_lib._lib.MoeAdamwConfig(**kw)
    assert lib.moe_adamw(ctypes.byref(c), adam_table(moe_lib), 1, None, None, P, None) == moe_lib.MOE_ERR_INVALID_ARG


def test_adamw_refuses_arrays(moe_lib):
    lib, c, inval = moe_lib.load(), moe_lib._lib.MoeAdamwConfig(1e-3, 0.9, 0.999, 1e-8), moe_lib.MOE_ERR_INVALID_ARG
    t = adam_table(moe_lib)
    assert lib.moe_adamw(None, t, 1, None, None, P, None) == inval
    assert lib.moe_adamw(ctypes.byref(c), None, 1, None, None, P, None) == inval
    assert lib.moe_adamw(ctypes.byref(c), t, -1, None, None, P, None) == inval
    for state in (None, ctypes.c_void_p(260)):
        assert lib.moe_adamw(ctypes.byref(c), t, 1, None, None, state, None) == inval
    assert lib.moe_adamw(ctypes.byref(c), t, 1, Q, None, P, None) == inval
    assert lib.moe_adamw(ctypes.byref(c), t, 1, None, Q, P, None) == inval


def test_binding_refuses_tensors(moe_lib):
    moe = moe_lib
    c = moe.make_embed_config(4, 6, 8)
    ids, W, y = torch.zeros(4, dtype=torch.int32), torch.zeros(6, 8).bfloat16(), torch.zeros(4, 8).bfloat16()
    for bad in ((ids.long(), W, y), (ids, W.float(), y), (ids, W, y.t()), (ids[:3], W, y)):
        with pytest.raises(ValueError):
            moe.embed(c, *bad)
    with pytest.raises(ValueError):
        moe.embed_backward(c, ids, y, W, torch.zeros(16, dtype=torch.uint8))
    c = moe.make_policy_config(4, 6)
    z, f, one = torch.zeros(4, 6).bfloat16(), torch.zeros(4), torch.zeros(1)
    with pytest.raises(ValueError):
        moe.token_logp(c, torch.zeros(4, 8).bfloat16()[:, :6], ids, f)      # rows 8 apart, ld says 6
    with pytest.raises(ValueError):
        moe.policy_loss(c, z, ids, f, f, None, f.double(), f, one, None, torch.zeros(4096))
    with pytest.raises(ValueError):
        moe.policy_loss(c, z, ids, f, f, None, f, f, one, None, None)       # loss without a workspace
    p = torch.zeros(300)
    with pytest.raises(ValueError):
        moe.AdamW([dict(p=p.half(), g=p)])
    with pytest.raises(ValueError):
        moe.AdamW([dict(p=p, g=p[:-1])])
    with pytest.raises(ValueError):
        moe.AdamW([dict(p=p, g=p, m=p.clone())])
    with pytest.raises(ValueError):
        moe.AdamW([dict(p=p, g=p, m=p.clone(), v=p.clone(), m_scale=torch.zeros(2), v_scale=torch.zeros(2))])
    with pytest.raises(ValueError):
        moe.AdamW([dict(p=p, g=p)], bits=16)
    opt = moe.AdamW([dict(p=p, g=p.clone())], bits=8, step=7)
    assert opt.tensors[0]["m"].dtype == torch.float8_e4m3fn and opt.tensors[0]["m_scale"].numel() == 2
    assert opt.steps_done() == 7 and abs(float(opt.state[0]) - (1 - 0.9 ** 7)) < 1e-15
    with pytest.raises(ValueError):
        opt.step(lr=torch.zeros(2))


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
def test_calls_without_gpu_report_cuda_error(moe_lib):
    lib = moe_lib.load()
    c = embed_cfg(moe_lib)
    assert lib.moe_embed(ctypes.byref(c), P, P, P, None) == moe_lib.MOE_ERR_CUDA
    assert lib.moe_embed_backward(ctypes.byref(c), P, P, P, P, None) == moe_lib.MOE_ERR_CUDA
    c = policy_cfg(moe_lib)
    assert lib.moe_policy_loss(ctypes.byref(c), *[P] * 8, ctypes.c_void_p(4096), P, None) == moe_lib.MOE_ERR_CUDA
    a = moe_lib._lib.MoeAdamwConfig(1e-3, 0.9, 0.999, 1e-8)
    assert lib.moe_adamw(ctypes.byref(a), adam_table(moe_lib), 1, None, None, P, None) == moe_lib.MOE_ERR_CUDA
