"""Policy loss, its gradient and token log-probabilities against the fp64 oracle.

Tolerances. x = z / tau has the range R over a row. The exponent (x - max) is a product with a
rounded constant: off by 2^-22 (1 + R) at most, and so is its exponential, which adds 2^-22 of
its own; a sum of V terms in fp32 over at least 256 threads is off by (V / 256 + 64) 2^-24; the
logarithm and its products by 2^-22 (1 + log V). Together tol_lp = 2^-22 (4 + 2 R + log V) +
2^-24 (V / 256 + 64), absolute, on logp. A gradient element is w / tau * slope * (1[target] - p):
the slope's parts A r and kl (1 - e^u) are off by 2 tol_lp of their size (old and ref enter a
difference with logp), p by 2 tol_lp of itself, and the result is rounded once to its type: by
half a step of it, which below the type's normal range is LEAST."""
import math

import numpy as np
import pytest
import torch

from oracle import train_oracle as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
LEAST = {"bf16": 2.0 ** -134, "f32": 2.0 ** -150}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(T, V, dtype, tau=1.0, lo=0.2, hi=0.2, seed=0, pad_ld=0):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(T, V, generator=g) * 2.5).to(DT[dtype])
    target = torch.randint(0, V, (T,), generator=g)
    z[torch.arange(T), target] += (torch.rand(T, generator=g) < 0.5).to(z.dtype) * 8
    lp = O.log_softmax_at(f64(z), target.numpy(), tau)
    lr = torch.randn(T, generator=g, dtype=torch.float64).numpy() * 0.2
    for border in (math.log(max(1 - lo, 1e-9)), math.log(1 + hi)):    # a border has two right gradients
        lr = np.where(np.abs(lr - border) < 1e-3, lr + 3e-3, lr)
    out = dict(z=z.cuda(), target=target.int().cuda(), old=torch.tensor(lp - lr).float().cuda(),
               ref=torch.tensor(lp).float().cuda() + 0.2 * torch.randn(T, generator=g).cuda(),
               adv=torch.randn(T, generator=g).cuda(), w=torch.rand(T, generator=g).cuda() + 0.5)
    if pad_ld:
        wide = torch.full((T, V + pad_ld), float("nan"), dtype=DT[dtype], device="cuda")
        wide[:, :V] = out["z"]
        out["z"] = wide[:, :V]
    return out


def tol_lp(z, tau, V):
    x = np.where(np.isfinite(z), z, 0) / tau
    R = x.max() - x.min()
    return 2.0 ** -22 * (4 + 2 * R + math.log(V)) + 2.0 ** -24 * (V / 256 + 64)


def check(moe, s, dtype, tau=1.0, lo=0.2, hi=0.2, kl=0.1, ld_grad=None, in_place=False, old=True, weight=True):
    z = s["z"]
    T, V = z.shape
    ld = z.stride(0) if T > 1 else max(V, z.stride(0))
    if in_place:
        ld_grad = ld
    c = moe.make_policy_config(T, V, dtype, tau, lo, hi, kl, ld, ld_grad)
    ref = O.policy(f64(z), s["target"].cpu().numpy(), f64(s["adv"]), f64(s["old"]) if old else None, f64(s["ref"]),
                   f64(s["w"]) if weight else None, np.float64(np.float32(tau)), np.float64(np.float32(lo)),
                   np.float64(np.float32(hi)), np.float64(np.float32(kl)))
    lp, loss = torch.full((T,), 9.0, device="cuda"), torch.full((1,), 9.0, device="cuda")
    if in_place:
        buf = torch.empty(T * ld + 16, dtype=DT[dtype], device="cuda")
        dz = z = buf.as_strided((T, V), (ld, 1)).copy_(z)
    else:
        buf = torch.full(((T - 1) * c.ld_grad + V + 64,), 5.0, dtype=DT[dtype], device="cuda")
        dz = buf.as_strided((T, V), (c.ld_grad, 1))
    ws = torch.full((moe.policy_workspace_bytes(c),), 0xFF, dtype=torch.uint8, device="cuda")
    moe.policy_loss(c, z, s["target"], s["adv"], s["old"] if old else None, s["ref"] if kl else None,
                    s["w"] if weight else None, lp, loss, dz, ws)
    w = np.abs(f64(s["w"])) if weight else np.ones(T)
    tl = tol_lp(f64(s["z"]), tau, V)
    k = ref["kept"]
    assert (np.abs(f64(lp) - ref["logp"]) <= tl + np.abs(ref["logp"]) * 2.0 ** -23).all()
    unit = np.where(k, w, 0) / tau * ref["size"]
    p = np.zeros_like(ref["dz"])
    if k.any():
        x = f64(s["z"])[k] / tau
        p[k] = np.exp(x - x.max(1, keepdims=True))
        p[k] /= p[k].sum(1, keepdims=True)
    hot = np.zeros_like(p)
    hot[np.flatnonzero(k), s["target"].cpu().numpy()[k]] = 1
    tol = unit[:, None] * (p + hot) * (4 * tl + 2.0 ** -21) + np.abs(ref["dz"]) * HALF[dtype] * 1.01 + LEAST[dtype] + 1e-44
    err = np.abs(f64(dz) - ref["dz"])
    assert (err <= tol).all(), (err - tol).max()
    assert (f64(dz)[~k] == 0).all()
    # each token's term is off by its slope times tol_lp, and by the rounding of its parts; the sum by its depth
    terms = np.abs(ref["tok"])
    assert abs(float(loss) - ref["loss"]) <= (np.where(k, w, 0) * (ref["size"] + abs(kl))).sum() * (2 * tl + 2.0 ** -20) \
        + terms.sum() * (T / 1024 + 16) * 2.0 ** -24
    if not in_place and ld_grad and ld_grad > V and T > 1:
        assert (buf.as_strided((T - 1, ld_grad - V), (ld_grad, 1), V) == 5).all()   # between the rows
    if not in_place:
        again = torch.empty_like(buf).as_strided(dz.shape, dz.stride())
        moe.policy_loss(c, z, s["target"], s["adv"], s["old"] if old else None, s["ref"] if kl else None,
                        s["w"] if weight else None, None, None, again, None)
        assert torch.equal(again, dz)                                               # bit for bit
        moe.policy_loss(c, z, s["target"], s["adv"], s["old"] if old else None, s["ref"] if kl else None,
                        s["w"] if weight else None, None, loss2 := torch.empty_like(loss), None, ws)
        assert torch.equal(loss, loss2)                                             # loss alone
    return lp, loss, dz


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(1, 1), (1, 2), (2, 7), (5, 8), (3, 37), (1, 1000), (17, 513), (9, 4099), (4, 33000),
                                 (2, 70001), (1, 131072), (1, 140001), (700, 300)])
def test_policy(T, V, dtype, moe_lib, cuda_device):
    check(moe_lib, make(T, V, dtype), dtype)
    moe_lib.get_error()


@pytest.mark.parametrize("T,V", [(400, 20001), (160, 65536), (330, 50021), (310, 131000)])
def test_policy_more_rows_than_sms(T, V, moe_lib, cuda_device):
    check(moe_lib, make(T, V, "bf16"), "bf16")


@pytest.mark.parametrize("dtype,V", [("bf16", 393216), ("bf16", 393300), ("bf16", 600001), ("f32", 196608), ("f32", 250003)])
def test_policy_rows_past_shared_memory(dtype, V, moe_lib, cuda_device):
    """The longest rows that a cluster keeps, and longer ones; also in place."""
    check(moe_lib, make(3, V, dtype), dtype)
    check(moe_lib, make(3, V, dtype), dtype, in_place=True)


@pytest.mark.parametrize("V", [300, 20001, 131072, 600001])
def test_token_logp_has_the_bits_of_the_loss(V, moe_lib, cuda_device):
    """Log-probabilities kept from token_logp give a ratio of exactly one."""
    s = make(40, V, "bf16")
    c = moe_lib.make_policy_config(40, V)
    a, b = torch.empty(40, device="cuda"), torch.empty(40, device="cuda")
    moe_lib.token_logp(c, s["z"], s["target"], a)
    moe_lib.policy_loss(c, s["z"], s["target"], s["adv"], a, None, None, b, None, torch.empty_like(s["z"]), None)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kl,old,weight,tau,lo,hi", [(0.0, True, True, 1.0, 0.2, 0.2), (0.1, False, True, 0.7, 0.2, 0.3),
                                                     (0.1, True, False, 1.3, 0.1, 0.4), (0.0, False, False, 2.0, 1.0, 0.0),
                                                     (-0.05, True, True, 0.25, 0.0, 5.0)])
def test_policy_settings(kl, old, weight, tau, lo, hi, dtype, moe_lib, cuda_device):
    check(moe_lib, make(40, 777, dtype, tau, lo, hi), dtype, tau, lo, hi, kl, old=old, weight=weight)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,pad,ld_grad", [(1000, 0, None), (1000, 24, 1024), (1001, 7, 1008), (1001, 0, 1003),
                                           (1003, 5, 1003), (64, 1, 65), (30011, 5, 30011), (30011, 5, 30016)])
def test_policy_strides_and_alignments(V, pad, ld_grad, dtype, moe_lib, cuda_device):
    s = make(6, V, dtype, pad_ld=pad)
    check(moe_lib, s, dtype, ld_grad=ld_grad)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,pad", [(5, 1000, 0), (3, 1001, 6), (2, 70001, 0), (300, 40003, 0), (1, 9, 0)])
def test_policy_in_place(T, V, pad, dtype, moe_lib, cuda_device):
    s = make(T, V, dtype, pad_ld=pad)
    check(moe_lib, s, dtype, in_place=True)


@pytest.mark.parametrize("V", [50, 5003, 90001])
def test_left_out_tokens(V, moe_lib, cuda_device):
    """Weight 0 or a negative target: nothing of the row is read, whatever it holds."""
    s = make(8, V, "bf16")
    s["w"][2] = 0
    s["w"][3] = -0.0
    s["target"][5] = -1
    s["target"][6] = -100
    clean = check(moe_lib, s, "bf16")
    for t, bad in ((2, float("nan")), (3, float("inf")), (5, float("nan")), (6, -float("inf"))):
        s["z"][t] = bad
    s["adv"][2] = s["old"][2] = s["ref"][2] = float("nan")
    T = 8
    c = moe_lib.make_policy_config(T, V, kl_weight=0.1)
    lp, loss, dz = torch.empty(T, device="cuda"), torch.empty(1, device="cuda"), torch.empty_like(s["z"])
    ws = torch.empty(moe_lib.policy_workspace_bytes(c), dtype=torch.uint8, device="cuda")
    moe_lib.policy_loss(c, s["z"], s["target"], s["adv"], s["old"], s["ref"], s["w"], lp, loss, dz, ws)
    for got, want in zip((lp, loss, dz), clean):
        assert torch.equal(got, want)
    s["w"].zero_()                                    # a batch with nothing in it
    moe_lib.policy_loss(c, s["z"], s["target"], s["adv"], s["old"], s["ref"], s["w"], lp, loss, dz, ws)
    assert float(loss) == 0 and (dz == 0).all() and (lp == 0).all()
    moe_lib.get_error()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [64, 4001, 80003])
def test_forbidden_tokens(V, dtype, moe_lib, cuda_device):
    """Logits of -inf, and of the type's lowest value, have probability 0 and gradient 0; a row may
    hold one token that is left."""
    s = make(5, V, dtype)
    t = s["target"].long()
    for row, low in ((0, -float("inf")), (1, torch.finfo(DT[dtype]).min), (2, -float("inf"))):
        mask = torch.rand(V, device="cuda") < 0.7
        if row == 2:
            mask[:] = True
        mask[t[row]] = False
        s["z"][row, mask] = low
    # log-probabilities moved: put the references where the oracle has them
    keep = f64(s["z"])
    keep[keep < -1e30] = -1e30
    lp = O.log_softmax_at(keep, t.cpu().numpy(), 1.0)
    s["old"], s["ref"] = torch.tensor(lp - 0.05).float().cuda(), torch.tensor(lp + 0.1).float().cuda()
    ref = O.policy(keep, t.cpu().numpy(), f64(s["adv"]), f64(s["old"]), f64(s["ref"]), f64(s["w"]), kl=np.float64(np.float32(0.1)))
    c = moe_lib.make_policy_config(5, V, dtype, kl_weight=0.1)
    got, loss, dz = torch.empty(5, device="cuda"), torch.empty(1, device="cuda"), torch.empty_like(s["z"])
    ws = torch.empty(moe_lib.policy_workspace_bytes(c), dtype=torch.uint8, device="cuda")
    moe_lib.policy_loss(c, s["z"], s["target"], s["adv"], s["old"], s["ref"], s["w"], got, loss, dz, ws)
    live = np.where(keep > -1e29, keep, 0)
    tl = tol_lp(live, 1.0, V)
    assert (np.abs(f64(got) - ref["logp"]) <= tl + 2.0 ** -23 * np.abs(ref["logp"])).all()
    assert float(got[2]) == 0.0                       # the only token left
    size = (f64(s["w"]) * ref["size"])[:, None]
    assert (np.abs(f64(dz) - ref["dz"]) <= size * 2 * (4 * tl + 2.0 ** -21) + np.abs(ref["dz"]) * HALF[dtype] * 1.01).all()
    assert (f64(dz)[keep < -1e29] == 0).all()


@pytest.mark.parametrize("V", [40, 5001, 100003])
@pytest.mark.parametrize("bad", ["none", "nan", "inf"])
def test_rows_without_a_distribution(V, bad, moe_lib, cuda_device):
    """-inf everywhere, a NaN or a +inf in a row: NaN there and in the loss, and in no other row."""
    s = make(6, V, "bf16")
    clean = check(moe_lib, s, "bf16")
    if bad == "none":
        s["z"][3] = -float("inf")
    else:
        s["z"][3, V // 3] = float(bad)
    c = moe_lib.make_policy_config(6, V, kl_weight=0.1)
    lp, loss, dz = torch.empty(6, device="cuda"), torch.empty(1, device="cuda"), torch.empty_like(s["z"])
    ws = torch.empty(moe_lib.policy_workspace_bytes(c), dtype=torch.uint8, device="cuda")
    moe_lib.policy_loss(c, s["z"], s["target"], s["adv"], s["old"], s["ref"], s["w"], lp, loss, dz, ws)
    assert lp[3].isnan() and loss.isnan().all() and dz[3].isnan().all()
    others = [0, 1, 2, 4, 5]
    assert torch.equal(lp[others], clean[0][others]) and torch.equal(dz[others], clean[2][others])


def test_target_of_probability_zero(moe_lib, cuda_device):
    """logp = -inf, ratio 0; the KL term is infinite, and without it all is finite."""
    s = make(3, 300, "f32")
    s["z"][1, s["target"][1].long()] = -float("inf")
    for kl in (0.0, 0.1):
        c = moe_lib.make_policy_config(3, 300, "f32", kl_weight=kl)
        lp, loss, dz = torch.empty(3, device="cuda"), torch.empty(1, device="cuda"), torch.empty_like(s["z"])
        ws = torch.empty(moe_lib.policy_workspace_bytes(c), dtype=torch.uint8, device="cuda")
        moe_lib.policy_loss(c, s["z"], s["target"], s["adv"], s["old"], s["ref"], s["w"], lp, loss, dz, ws)
        assert float(lp[1]) == -float("inf")
        assert (float(loss) == float("inf")) if kl else bool(loss.isfinite().all() and (dz[1] == 0).all())
        assert dz[[0, 2]].isfinite().all()


def test_bad_targets_are_reported_and_left_out(moe_lib, cuda_device):
    s = make(5, 100, "bf16")
    want = check(moe_lib, s, "bf16")[2].clone()
    s["target"][1] = 100
    s["target"][3] = 2 ** 31 - 1
    got = check(moe_lib, s, "bf16")[2]
    with pytest.raises(moe_lib.MoeError) as e:
        moe_lib.get_error()
    assert e.value.status == moe_lib.MOE_ERR_DEVICE_BOUNDS
    assert (got[[1, 3]] == 0).all() and torch.equal(got[[0, 2, 4]], want[[0, 2, 4]])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,tau,pad", [(1, 1, 1.0, 0), (1, 131072, 0.7, 0), (4, 131071, 1.0, 0), (3, 99, 1.0, 2),
                                         (500, 700, 0.5, 0), (200, 32000, 1.0, 3)])
def test_token_logp(T, V, tau, pad, dtype, moe_lib, cuda_device):
    s = make(T, V, dtype, tau, pad_ld=pad)
    c = moe_lib.make_policy_config(T, V, dtype, tau, ld=V + pad)
    lp = torch.empty(T, device="cuda")
    moe_lib.token_logp(c, s["z"], s["target"], lp)
    ref = O.log_softmax_at(f64(s["z"]), s["target"].cpu().numpy(), np.float64(np.float32(tau)))
    assert (np.abs(f64(lp) - ref) <= tol_lp(f64(s["z"]), tau, V) + np.abs(ref) * 2.0 ** -23).all()
    s["target"][T // 2] = -1
    moe_lib.token_logp(c, s["z"], s["target"], lp)
    assert float(lp[T // 2]) == 0
    moe_lib.get_error()


@pytest.mark.parametrize("V", [300, 20001])
def test_token_logp_with_a_loss_configuration(V, moe_lib, cuda_device):
    """The loss's own configuration, KL term and clipping set: token_logp has no reference to read."""
    s = make(20, V, "bf16")
    a, b = torch.empty(20, device="cuda"), torch.empty(20, device="cuda")
    moe_lib.token_logp(moe_lib.make_policy_config(20, V), s["z"], s["target"], a)
    moe_lib.token_logp(moe_lib.make_policy_config(20, V, clip_low=0.1, kl_weight=0.3), s["z"], s["target"], b)
    assert torch.equal(a, b)


def test_large_logits_lose_nothing(moe_lib, cuda_device):
    """Logits around 3e4: the log-probability of their differences, as for the same row around 0."""
    z = torch.randn(4, 3001, generator=torch.Generator().manual_seed(3)).mul(64).round().div(16).cuda()
    t = torch.tensor([0, 7, 1500, 3000], dtype=torch.int32, device="cuda")
    c, a, b = moe_lib.make_policy_config(4, 3001, "f32"), torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    moe_lib.token_logp(c, z, t, a)
    moe_lib.token_logp(c, z + 32768.0, t, b)
    ref = O.log_softmax_at(f64(z), t.cpu().numpy(), 1.0)
    assert (np.abs(f64(a) - ref) <= tol_lp(f64(z), 1.0, 3001) + np.abs(ref) * 2.0 ** -23).all()
    assert torch.equal(a, b)                          # sixteenths: every difference is exact


def test_empty_batch(moe_lib, cuda_device):
    c = moe_lib.make_policy_config(0, 100)
    e, z = torch.empty(0, device="cuda"), torch.empty(0, 100, device="cuda").bfloat16()
    loss = torch.ones(1, device="cuda")
    ws = torch.empty(moe_lib.policy_workspace_bytes(c), dtype=torch.uint8, device="cuda")
    moe_lib.policy_loss(c, z, e.int(), e, e, None, e, e, loss, z.clone(), ws)
    moe_lib.token_logp(c, z, e.int(), e)
    assert float(loss) == 0


def test_rows_past_two_billion_elements(moe_lib, cuda_device):
    s = make(3, 1000, "bf16")
    ld = 2 ** 30 + 3
    for in_place in (True, False):
        wide = torch.empty(2 * ld + 1000, dtype=torch.bfloat16, device="cuda").as_strided((3, 1000), (ld, 1))
        wide.copy_(s["z"])
        c = moe_lib.make_policy_config(3, 1000, ld=ld, ld_grad=ld if in_place else None)
        dz = wide if in_place else torch.empty(3, 1000, dtype=torch.bfloat16, device="cuda")
        small = moe_lib.make_policy_config(3, 1000)
        want = torch.empty(3, 1000, dtype=torch.bfloat16, device="cuda")
        moe_lib.policy_loss(small, s["z"], s["target"], s["adv"], s["old"], None, s["w"], None, None, want, None)
        moe_lib.policy_loss(c, wide, s["target"], s["adv"], s["old"], None, s["w"], None, None, dz, None)
        ref = O.policy(f64(s["z"]), s["target"].cpu().numpy(), f64(s["adv"]), f64(s["old"]), None, f64(s["w"]))
        # the rows' alignments differ, and with them the order of sums
        assert (np.abs(f64(dz) - ref["dz"]) <= 1e-4 * np.abs(ref["dz"]).max() + np.abs(ref["dz"]) * 2.0 ** -8).all()
        assert (np.abs(f64(want) - ref["dz"]) <= 1e-4 * np.abs(ref["dz"]).max() + np.abs(ref["dz"]) * 2.0 ** -8).all()


def test_other_stream_and_graph(moe_lib, cuda_device):
    s = make(30, 9001, "bf16")
    c = moe_lib.make_policy_config(30, 9001, kl_weight=0.1)
    ws = torch.empty(moe_lib.policy_workspace_bytes(c), dtype=torch.uint8, device="cuda")

    def call(lp, loss, dz, st=None):
        moe_lib.policy_loss(c, s["z"], s["target"], s["adv"], s["old"], s["ref"], s["w"], lp, loss, dz, ws, st)

    def outs():
        return torch.empty(30, device="cuda"), torch.empty(1, device="cuda"), torch.empty_like(s["z"])

    a, b = outs(), outs()
    call(*a)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        call(*b, st)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    s["adv"].neg_()
    graph.replay()
    call(*a)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
