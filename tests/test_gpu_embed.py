"""Token embedding and its gradient against the fp64 oracle.

Tolerances count roundings: the lookup is one fp32 product and one rounding to the output type;
an element of the gradient is a sum of n terms in fp32 (at most n additions, one product by the
scale, one addition to what was there), each off by 2^-24 of the running magnitude, then one
rounding to the output type."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def f64(t):
    return t.detach().double().cpu().numpy()


def make(T, V, d, dtype, seed=0, tokens="zipf"):
    g = torch.Generator().manual_seed(seed)
    if tokens == "zipf":
        ids = (torch.rand(T, generator=g, dtype=torch.float64).pow(4) * V).long().clamp(max=V - 1)
    elif tokens == "same":
        ids = torch.full((T,), V // 2)
    else:
        ids = torch.randperm(V, generator=g)[:T]
    W = torch.randn(V, d, generator=g).to(DT[dtype])
    dy = torch.randn(T, d, generator=g).to(DT[dtype])
    return ids.int().cuda(), W.cuda(), dy.cuda()


def check_forward(moe, ids, W, scale, dtype):
    T, (V, d) = len(ids), W.shape
    c = moe.make_embed_config(T, V, d, scale=scale, dtype=dtype)
    y = torch.full((T, d), float("nan"), dtype=DT[dtype], device="cuda")
    moe.embed(c, ids, W, y)
    ref = O.embed(ids.cpu().numpy(), f64(W), np.float64(np.float32(scale)))
    assert (np.abs(f64(y) - ref) <= np.abs(ref) * (HALF[dtype] + 2.0 ** -24) * 1.001).all()
    return y


def check_backward(moe, ids, dy, V, scale, dtype, grad, accumulate, pad, seed=0):
    T, d = dy.shape
    c = moe.make_embed_config(T, V, d, scale=scale, dtype=dtype, grad_dtype=grad, accumulate=accumulate,
                              padding_id=pad)
    g = torch.Generator().manual_seed(seed + 1)
    dW0 = torch.randn(V, d, generator=g).to(DT[grad]).cuda() if accumulate else \
        torch.full((V, d), float("nan"), dtype=DT[grad], device="cuda")
    ws = torch.full((moe.embed_workspace_bytes(c),), 0xAB, dtype=torch.uint8, device="cuda")
    dW = dW0.clone()
    moe.embed_backward(c, ids, dy, dW, ws)
    ref, mag, n = O.embed_backward(ids.cpu().numpy(), f64(dy), V, np.float64(np.float32(scale)), pad,
                                   f64(dW0) if accumulate else None)
    tol = (n[:, None] + 3) * 2.0 ** -24 * mag + np.abs(ref) * HALF[grad] * 1.001
    got = f64(dW)
    assert (np.abs(got - ref) <= tol).all(), np.abs(got - ref).max()
    if accumulate:      # rows of tokens that do not occur are not touched
        assert (got[n == 0] == f64(dW0)[n == 0]).all()
    else:
        assert (got[n == 0] == 0).all()
    again = dW0.clone()
    moe.embed_backward(c, ids, dy, again, ws)
    assert torch.equal(again, dW)                       # bit for bit
    moe.get_error()
    return dW


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,d", [(1, 1, 1), (1, 500, 1024), (3, 17, 37), (33, 100, 130), (257, 1000, 64),
                                   (1000, 33, 4), (2049, 5003, 1026)])
def test_lookup(T, V, d, dtype, moe_lib, cuda_device):
    ids, W, _ = make(T, V, d, dtype)
    check_forward(moe_lib, ids, W, 32.0, dtype)
    check_forward(moe_lib, ids, W, 0.3, dtype)
    moe_lib.get_error()


def test_lookup_long_batch(moe_lib, cuda_device):
    """Several vectors a thread."""
    ids, W, _ = make(40000, 300, 512, "bf16")
    check_forward(moe_lib, ids, W, 1.0, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(2001, 1021), (3001, 1022), (6001, 1020)])
def test_lookup_long_batch_of_short_vectors(T, d, dtype, moe_lib, cuda_device):
    """The same for rows of one, two and four elements a vector."""
    ids, W, _ = make(T, 100, d, dtype)
    check_forward(moe_lib, ids, W, 0.3, dtype)


@pytest.mark.parametrize("dtype,grad", [("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("T,V,d", [(1029, 300, 131), (1029, 4000, 131), (1029, 60, 262)])
def test_gradient_of_short_vectors(T, V, d, dtype, grad, accumulate, moe_lib, cuda_device):
    """Whole groups in flight: runs inside them, across them, and both."""
    ids, _, dy = make(T, V, d, dtype)
    check_backward(moe_lib, ids, dy, V, 0.7, dtype, grad, accumulate, pad=-1)


@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("T,V,d", [(1, 1, 1), (1, 700, 64), (31, 3, 37), (32, 40, 8), (33, 1000, 130), (257, 90, 6),
                                   (1025, 513, 100), (4500, 70000, 16)])
def test_gradient(T, V, d, dtype, grad, accumulate, moe_lib, cuda_device):
    ids, _, dy = make(T, V, d, dtype)
    check_backward(moe_lib, ids, dy, V, 8.0, dtype, grad, accumulate, pad=-1)
    check_backward(moe_lib, ids, dy, V, 1.0, dtype, grad, accumulate, pad=int(ids[0]))


@pytest.mark.parametrize("T", [5, 32, 33, 64, 100, 1024, 3000])
def test_gradient_of_one_token_repeated(T, moe_lib, cuda_device):
    """One run over all groups of rows: every length at which a run ends on or across a border."""
    ids, _, dy = make(T, 9, 72, "bf16", tokens="same")
    check_backward(moe_lib, ids, dy, 9, 1.0, "bf16", "f32", False, pad=-1)
    check_backward(moe_lib, ids, dy, 9, 1.0, "bf16", "f32", True, pad=4)     # all of them padding


def test_gradient_of_distinct_tokens(moe_lib, cuda_device):
    ids, _, dy = make(1500, 1500, 64, "bf16", tokens="perm")
    dW = check_backward(moe_lib, ids, dy, 1500, 1.0, "bf16", "bf16", False, pad=-1)
    assert torch.equal(dW[ids.long()], dy)                # nothing to add: exactly the rows


@pytest.mark.parametrize("V", [511, 512, 513, 262143, 262144, 300000])
def test_gradient_vocabulary_sizes(V, moe_lib, cuda_device):
    """Around the borders of the sort's digits (the key V itself marks what is left out)."""
    g = torch.Generator().manual_seed(V)
    ids = torch.randint(max(0, V - 700), V, (900,), generator=g).int()
    ids[:3] = torch.tensor([0, V - 1, V - 1], dtype=torch.int32)
    dy = torch.randn(900, 8, generator=g).cuda()
    check_backward(moe_lib, ids.cuda(), dy, V, 1.0, "f32", "f32", False, pad=V - 1)


@pytest.mark.parametrize("T", [1023, 1024, 16383, 16384, 16385, 70001])
def test_many_chunks(T, moe_lib, cuda_device):
    """Around the sizes at which the sort takes one more pair a thread, or more than one block."""
    ids, _, dy = make(T, 3001, 24, "bf16")
    check_backward(moe_lib, ids, dy, 3001, 1.0, "bf16", "f32", False, pad=0)
    check_backward(moe_lib, ids, dy, 3001, 1.0, "bf16", "bf16", True, pad=-1)


@pytest.mark.parametrize("T,V,d", [(16384, 262145, 8), (5000, 400000, 4), (20000, 1, 3)])
def test_gradient_more_vocabularies(T, V, d, moe_lib, cuda_device):
    ids, _, dy = make(T, V, d, "f32")
    check_backward(moe_lib, ids, dy, V, 1.0, "f32", "f32", False, pad=-1)


def test_empty_batch(moe_lib, cuda_device):
    moe = moe_lib
    for acc in (False, True):
        c = moe.make_embed_config(0, 70, 24, accumulate=acc)
        ids, dy = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(0, 24, device="cuda").bfloat16()
        dW = torch.ones(70, 24, device="cuda").bfloat16()
        ws = torch.empty(moe.embed_workspace_bytes(c), dtype=torch.uint8, device="cuda")
        moe.embed(c, ids, dW.clone(), dy)
        moe.embed_backward(c, ids, dy, dW, ws)
        assert (dW == (1 if acc else 0)).all()
    moe.get_error()


def test_bad_ids_are_reported_and_left_out(moe_lib, cuda_device):
    moe = moe_lib
    ids, W, dy = make(300, 50, 40, "bf16")
    ids[7], ids[8], ids[299] = -1, 50, -2 ** 31
    y = check_forward(moe, ids, W, 2.0, "bf16")
    assert (y[[7, 8, 299]] == 0).all()
    with pytest.raises(moe.MoeError) as e:
        moe.get_error()
    assert e.value.status == moe.MOE_ERR_DEVICE_BOUNDS
    c = moe.make_embed_config(300, 50, 40, grad_dtype="f32")
    dW = torch.empty(50, 40, device="cuda")
    moe.embed_backward(c, ids, dy, dW, torch.empty(moe.embed_workspace_bytes(c), dtype=torch.uint8, device="cuda"))
    with pytest.raises(moe.MoeError) as e:
        moe.get_error()
    assert e.value.status == moe.MOE_ERR_DEVICE_BOUNDS
    ref, mag, n = O.embed_backward(ids.cpu().numpy(), f64(dy), 50, 1.0)
    assert (np.abs(f64(dW) - ref) <= (n[:, None] + 3) * 2.0 ** -24 * mag + np.abs(ref) * 2.0 ** -24).all()
    moe.get_error()


def test_nan_rows_stay_where_they_are(moe_lib, cuda_device):
    """A NaN in the row of a padding token reaches nothing; one in a token's row reaches that row alone."""
    moe = moe_lib
    ids = torch.tensor([1, 2, 0, 2, 3, 0], dtype=torch.int32, device="cuda")
    dy = torch.ones(6, 16, device="cuda")
    dy[2], dy[5], dy[1, 3] = float("nan"), float("inf"), float("nan")
    c = moe.make_embed_config(6, 5, 16, dtype="f32", padding_id=0)
    dW = torch.empty(5, 16, device="cuda")
    moe.embed_backward(c, ids, dy, dW, torch.empty(moe.embed_workspace_bytes(c), dtype=torch.uint8, device="cuda"))
    want = torch.zeros(5, 16)
    want[1], want[2], want[3], want[2, 3] = 1, 2, 1, float("nan")
    assert torch.equal(dW.cpu().nan_to_num(-7), want.nan_to_num(-7))


def test_gradient_against_differences(moe_lib, cuda_device):
    """d/dW of sum(y * dy), along random directions, in fp32: the loss is linear in W."""
    moe = moe_lib
    ids, W, dy = make(200, 30, 20, "f32")
    c = moe.make_embed_config(200, 30, 20, scale=1.5, dtype="f32")
    dW, y = torch.empty_like(W), torch.empty(200, 20, device="cuda")
    moe.embed_backward(c, ids, dy, dW, torch.empty(moe.embed_workspace_bytes(c), dtype=torch.uint8, device="cuda"))
    g = torch.Generator().manual_seed(5)
    for _ in range(4):
        D = torch.randn(30, 20, generator=g).cuda()
        moe.embed(c, ids, D, y)
        a, b = (y.double() * dy.double()).sum().item(), (D.double() * dW.double()).sum().item()
        size = (y.double() * dy.double()).abs().sum().item()
        assert abs(a - b) <= size * 210 * 2.0 ** -24


def test_rows_past_two_billion_elements(moe_lib, cuda_device):
    """Element offsets that pass 32 bits."""
    moe = moe_lib
    V, d = 1_100_000, 2048
    W = torch.empty(V, d, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([0, V - 1, V // 2, V - 1], dtype=torch.int32, device="cuda")
    W[ids.long()] = torch.randn(4, d, device="cuda").bfloat16()
    c = moe.make_embed_config(4, V, d)
    y = torch.empty(4, d, dtype=torch.bfloat16, device="cuda")
    moe.embed(c, ids, W, y)
    assert torch.equal(y, W[ids.long()])
    dy = torch.randn(4, d, device="cuda").bfloat16()
    W.fill_(7)
    moe.embed_backward(c, ids, dy, W, torch.empty(moe.embed_workspace_bytes(c), dtype=torch.uint8, device="cuda"))
    assert torch.equal(W[0], dy[0]) and torch.equal(W[V // 2], dy[2])
    assert torch.equal(W[V - 1], (dy[1].float() + dy[3].float()).bfloat16())
    assert int(torch.count_nonzero(W.view(torch.int16).sum(1, dtype=torch.int64))) <= 3
    moe.get_error()


def test_other_stream_and_graph(moe_lib, cuda_device):
    """On a stream of its own, and captured: the same bits; the graph follows ids refilled in place."""
    moe = moe_lib
    ids, W, dy = make(700, 900, 96, "bf16")
    c = moe.make_embed_config(700, 900, 96, grad_dtype="f32")
    ws = torch.empty(moe.embed_workspace_bytes(c), dtype=torch.uint8, device="cuda")
    y, dW = torch.empty_like(dy), torch.empty(900, 96, device="cuda")
    moe.embed(c, ids, W, y)
    moe.embed_backward(c, ids, dy, dW, ws)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y2, dW2 = torch.empty_like(y), torch.empty_like(dW)
    moe.embed(c, ids, W, y2, s)
    moe.embed_backward(c, ids, dy, dW2, ws, s)
    s.synchronize()
    assert torch.equal(y, y2) and torch.equal(dW, dW2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        moe.embed(c, ids, W, y2, s)
        moe.embed_backward(c, ids, dy, dW2, ws, s)
    ids.copy_(ids.flip(0))
    graph.replay()
    moe.embed(c, ids, W, y)
    moe.embed_backward(c, ids, dy, dW, torch.empty_like(ws))
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(dW, dW2)
    moe.get_error()
