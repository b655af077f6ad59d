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
