"""Embedding and its gradient on batches of millions of tokens and more."""
import pytest
import torch

from oracle import train_oracle as O

pytestmark = pytest.mark.gpu


def grad_call(moe, T, V, d, seed=0, accumulate=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    dy = torch.randint(-4, 5, (T, d), generator=g, device="cuda", dtype=torch.int32).bfloat16()
    cfg = moe.make_embed_config(T, V, d, grad_dtype="f32", accumulate=accumulate)
    dW = torch.full((V, d), 3.0, device="cuda")
    ws = torch.empty(moe.embed_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    return ids, dy, dW, lambda: moe.embed_backward(cfg, ids, dy, dW, ws)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("T,V,d", [(15360, 5003, 3), (15361, 5003, 3), (131072, 3, 8), (131073, 70001, 8), (1000003, 300000, 1),
                                   (200000, 1, 2), (4194305, 50021, 4)])
def test_gradient_of_many_chunks(T, V, d, accumulate, moe_lib, cuda_device):
    """Around the size from which the digits' counts are scanned by a launch of their own. Small whole
    numbers: every sum is exact in fp32, in any order."""
    ids, dy, dW, call = grad_call(moe_lib, T, V, d, accumulate=accumulate)
    call()
    ref, _, _ = O.embed_backward(ids.cpu().numpy(), dy.double().cpu().numpy(), V, 1.0,
                                 dW0=None if not accumulate else torch.full((V, d), 3.0).numpy())
    assert torch.equal(dW.double().cpu(), torch.from_numpy(ref))
    moe_lib.get_error()


def test_time_grows_with_the_batch(moe_lib, cuda_device):
    """Four times the tokens take about four times as long, not sixteen."""
    took = []
    for T in (2 ** 22, 2 ** 24):
        _, _, _, call = grad_call(moe_lib, T, 50021, 1)
        call()
        a, b = (torch.cuda.Event(enable_timing=True) for _ in "ab")
        best = float("inf")
        for _ in range(3):
            a.record()
            call()
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        took.append(best)
    assert took[1] < 8 * took[0], took


def test_more_than_a_billion_tokens(moe_lib, cuda_device):
    """Positions past 2^30, keys of four digits, rows left for the last launch to zero. One in three
    tokens carries a one: each row of the gradient is a count, exact in fp32; odd ids do not occur."""
    moe = moe_lib
    T, V = 2 ** 30 + 4097, 2 ** 27 + 5
    g = torch.Generator(device="cuda").manual_seed(0)
    ids = torch.randint(0, V // 2, (T,), generator=g, device="cuda", dtype=torch.int32).mul_(2)
    dy = torch.zeros(T, 1, dtype=torch.bfloat16, device="cuda")
    dy[::3] = 1
    cfg = moe.make_embed_config(T, V, 1, grad_dtype="f32")
    dW = torch.full((V, 1), float("nan"), device="cuda")
    ws = torch.empty(moe.embed_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    moe.embed_backward(cfg, ids, dy, dW, ws)
    moe.get_error()
    del ws, dy
    assert torch.equal(dW[:, 0], torch.bincount(ids[::3].long(), minlength=V).float())
    assert not dW[1::2].any()


def test_lookup_of_more_than_a_billion_vectors(moe_lib, cuda_device):
    """The vectors of one launch are numbered in 31 bits: a second launch takes the rest."""
    moe = moe_lib
    for T, d in ((2 ** 30 + 4097, 1), (2 ** 29 + 77, 3)):
        g = torch.Generator(device="cuda").manual_seed(T)
        W = torch.randn(1000, d, generator=g, device="cuda").bfloat16()
        ids = torch.randint(0, 1000, (T,), generator=g, device="cuda", dtype=torch.int32)
        y = torch.full((T, d), 9.0, dtype=torch.bfloat16, device="cuda")
        moe.embed(moe.make_embed_config(T, 1000, d), ids, W, y)
        for a in range(0, T, 2 ** 27):
            assert torch.equal(y[a:a + 2 ** 27], W[ids[a:a + 2 ** 27]])
    moe.get_error()
