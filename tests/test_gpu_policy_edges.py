"""Policy loss and token log-probabilities at the edges of rows: the elements before a row's first and
after its last whole 16-byte vector."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def masked_rows(T, V, dtype, seed=0):
    """Rows of -inf with eight finite logits, whose vectors belong to no thread that has an edge element;
    one of the eight is the target. An odd V starts the rows at every alignment."""
    g = torch.Generator().manual_seed(seed)
    n = 16 // (2 if dtype == "bf16" else 4)
    at = V // 2 // (256 * n) * 256 * n + 100 * n + torch.arange(8) if V > 2 * 256 * n else V // 2 + torch.arange(8)
    z = torch.full((T, V), -float("inf"))
    z[:, at] = torch.randn(T, 8, generator=g)
    target = at[torch.randint(0, 8, (T,), generator=g)]
    return z.to(DT[dtype]).cuda(), target.int().cuda()


@pytest.mark.parametrize("dtype,V", [("bf16", 301), ("bf16", 5003), ("bf16", 20001), ("bf16", 50257), ("bf16", 140003),
                                     ("bf16", 600001), ("f32", 303), ("f32", 9001), ("f32", 70003), ("f32", 250003)])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_edge_elements_of_masked_rows(dtype, V, bad, moe_lib, cuda_device):
    """A NaN or +inf in a row's first or last element, all but a few of the others being -inf: NaN for the
    row and the loss, and nothing for the other rows."""
    T = 17
    z, target = masked_rows(T, V, dtype)
    adv, old = torch.ones(T, device="cuda"), torch.full((T,), -2.0, device="cuda")
    cfg = moe_lib.make_policy_config(T, V, dtype)
    ws = torch.empty(moe_lib.policy_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")

    def call():
        lp, own, loss, dz = (torch.empty(*s, device="cuda", dtype=t) for s, t in
                             (((T,), torch.float32), ((T,), torch.float32), ((1,), torch.float32), ((T, V), DT[dtype])))
        moe_lib.policy_loss(cfg, z, target, adv, old, None, None, lp, loss, dz, ws)
        moe_lib.token_logp(cfg, z, target, own)
        return lp, own, loss, dz

    clean = call()
    assert all(x.isfinite().all() for x in clean)
    rows = {t: (0 if t % 2 else V - 1) for t in range(1, T, 2)} | {t: (V - 1 if t % 4 else 0) for t in range(2, T, 4)}
    for t, v in rows.items():
        z[t, v] = float(bad)
    lp, own, loss, dz = call()
    hit = torch.tensor(sorted(rows), device="cuda")
    rest = torch.tensor([t for t in range(T) if t not in rows], device="cuda")
    assert lp[hit].isnan().all() and own[hit].isnan().all() and loss.isnan().all() and dz[hit].isnan().all()
    for got, want in ((lp, clean[0]), (own, clean[1]), (dz, clean[3])):
        assert torch.equal(got[rest], want[rest])
    moe_lib.get_error()


@pytest.mark.parametrize("V", [2040, 40003])
def test_fp32_gradient_keeps_its_bits(V, moe_lib, cuda_device):
    """Probabilities of near logits, as quotients of two elements of one gradient row (which the row's sum
    and the token's factor do not enter). One is exp(z - top): a product with a rounded constant (2 of
    2^-24 of an exponent below 0.15), two fast exponentials (2^-22 each), two products, and as much less
    the exponent for the top: under 2^-21 + 8 * 2^-24 of itself."""
    g = torch.Generator().manual_seed(0)
    T = 6
    z = -torch.rand(T, V, generator=g) * 0.14
    z[:, 7] = 0.0
    z[:, 5] = 1.0e-3                                  # the target: the row's maximum, and no part of the quotients
    z = z.cuda()
    target = torch.full((T,), 5, dtype=torch.int32, device="cuda")
    dz = torch.empty_like(z)
    moe_lib.policy_loss(moe_lib.make_policy_config(T, V, "f32"), z, target, torch.ones(T, device="cuda"), None, None, None,
                        None, None, dz, None)
    got = dz.double() / dz[:, 7:8].double()
    off = (got / z.double().exp() - 1).abs()
    off[:, 5] = 0
    assert float(off.max()) <= 2.0 ** -21 + 8 * 2.0 ** -24


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_of_tiny_probabilities(dtype, moe_lib, cuda_device):
    """Probabilities from one down to below the least fp32 number, on a factor of 2^40: each element is
    right to its type's resolution, the normal range's end included."""
    V = 4 * 1001
    z = torch.linspace(0, -160, V).repeat(2, 1).to(DT[dtype]).cuda()
    target = torch.zeros(2, dtype=torch.int32, device="cuda")
    dz = torch.empty_like(z)
    adv = torch.tensor([1.0, 2.0 ** 40], device="cuda")
    moe_lib.policy_loss(moe_lib.make_policy_config(2, V, dtype), z, target, adv, None, None, None, None, None, dz, None)
    p = torch.softmax(z.double(), 1)
    p[:, 0] -= 1
    ref = p * adv.double()[:, None]
    half, least = (2.0 ** -8, 2.0 ** -134) if dtype == "bf16" else (2.0 ** -24, 2.0 ** -150)
    # the exponent, up to 231, has two roundings of 2^-24; the row's sum (over 256 threads and more) and the rest 2^-20
    tol = ref.abs() * (half * 1.01 + 2 * 231 * 2.0 ** -24 + 2.0 ** -20) + 2 * least + 2.0 ** -148
    assert ((dz.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(64, 300), (64, 5003), (300, 20001), (40, 131072), (5, 600001)])
def test_fresh_log_probabilities_give_a_ratio_of_one(T, V, dtype, moe_lib, cuda_device):
    """old_logp kept from token_logp of the same rows: the ratio is exactly one, so that with no room to
    clip (clip_low = clip_high = 0) no token loses its gradient, and everything is as on-policy."""
    g = torch.Generator(device="cuda").manual_seed(T)
    z = (torch.randn(T, V, generator=g, device="cuda") * 2.5).to(DT[dtype])
    target = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    adv = torch.randn(T, generator=g, device="cuda")
    cfg = moe_lib.make_policy_config(T, V, dtype, temperature=0.7, clip_low=0.0, clip_high=0.0)
    ws = torch.empty(moe_lib.policy_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    old = torch.empty(T, device="cuda")
    moe_lib.token_logp(cfg, z, target, old)
    got = []
    for o in (old, None):
        loss, dz = torch.empty(1, device="cuda"), torch.empty_like(z)
        moe_lib.policy_loss(cfg, z, target, adv, o, None, None, None, loss, dz, ws)
        got.append((loss, dz))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert (got[0][1][torch.arange(T, device="cuda"), target.long()] != 0).all()


def test_log_probabilities_of_another_batch_size(moe_lib, cuda_device):
    """The same row in a smaller batch may go over more blocks and be added up in another order: equal to
    rounding. A sum of 131072 exponentials over 256 threads and more: 576 roundings of 2^-24, the rest
    2^-22 (4 + ln V) and half a step of a number below 16."""
    V = 131072
    z = torch.randn(600, V, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    target = torch.arange(600, device="cuda", dtype=torch.int32)
    one = torch.empty(600, device="cuda")
    moe_lib.token_logp(moe_lib.make_policy_config(600, V), z, target, one)
    for T in (1, 7, 150, 599):
        lp = torch.empty(T, device="cuda")
        moe_lib.token_logp(moe_lib.make_policy_config(T, V), z[:T], target[:T], lp)
        assert float((lp - one[:T]).abs().max()) <= 576 * 2.0 ** -24 + 16 * 2.0 ** -22 + 2.0 ** -21


def test_low_part_of_a_log_probability_near_the_maximum(moe_lib, cuda_device):
    """A target a little below the maximum of a long, flat row: (z - max) is small beside ln(sum), and the
    rounding of their difference has to be kept all the same. The row's sum is a whole number but for
    the target's part (2^-24 of itself), the ratio's exponential is off by 2^-22, the gradient by three
    roundings of 2^-24: 2^-21 in all; a low part lost to the larger term's rounding is 2^-20."""
    V = 2 ** 24 + 2 ** 20
    low = torch.tensor([5343222, 5447694, 5088830, 1473506, 4542106, 674442, 2514166, 3382610], device="cuda") * 2.0 ** -21
    T = len(low)
    z = torch.zeros(T, V, device="cuda")
    target = torch.arange(T, device="cuda", dtype=torch.int32) * 999999
    z[torch.arange(T, device="cuda"), target.long()] = -low
    lp = -low.double() - torch.log(V - 1 + torch.exp(-low.double()))
    old = lp.float() + 2.0 ** -10
    want = torch.exp(lp - old.double())
    dz = torch.empty_like(z)
    cfg = moe_lib.make_policy_config(T, V, "f32", clip_low=1.0, clip_high=9.0)
    moe_lib.policy_loss(cfg, z, target, torch.full((T,), -1.0, device="cuda"), old, None, None, None, None, dz, None)
    got = dz[torch.arange(T, device="cuda"), target.long()].double() / (1 - lp.exp())
    assert float((got / want - 1).abs().max()) <= 2.0 ** -21
