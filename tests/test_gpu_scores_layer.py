"""The layer with its choice from scores, forward and backward, and the block around it: layer norm, gate,
scored choice, experts, and back, against automatic differentiation in 64 bits on the same choice.

Tolerances are the layer's parity tolerances (largest difference over the largest value: 2e-2 in bf16,
1e-4 in fp32)."""
import pytest
import torch

import parity as P

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TINY = 1e-20


def make(T, d, E, f, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)

    def r(*s, size=1.0):
        return (torch.randn(*s, generator=g) * size).to(DT[dtype])
    p = dict(Wg=r(E, d, size=d ** -0.5), W1=r(E, f, d, size=d ** -0.5), b1=r(E, f, size=0.1),
             W2=r(E, d, f, size=f ** -0.5), b2=r(E, d, size=0.1))
    p["bg"] = (torch.randn(E, generator=g) * 0.1)
    return p, r(T, d), r(T, d), torch.randn(E, generator=g) * 0.02


def gate64(z, idx, kind, renorm, scale, tau):
    x = z / tau
    s = torch.softmax(x, 1) if kind == "softmax" else torch.sigmoid(x)
    w = s.gather(1, idx)
    if renorm:
        w = w / (w.sum(1, keepdim=True) + (TINY if kind == "sigmoid" else 0))
    return scale * w


def layer64(x, p, idx, kept, gate, z_of=None):
    """y and z of the layer on the given choice; kept [T, k]: slots that were not dropped."""
    z = x @ p["Wg"].T + p["bg"]
    w = gate64(z, idx, *gate)
    y = torch.zeros_like(x)
    for e in range(p["Wg"].shape[0]):
        t, j = ((idx == e) & kept).nonzero(as_tuple=True)
        if len(t):
            h = torch.nn.functional.gelu(x[t] @ p["W1"][e].T + p["b1"][e])
            y = y.index_add(0, t, w[t, j][:, None] * (h @ p["W2"][e].T + p["b2"][e]))
    return y, z, w


def forward(moe, c, s, p, x, b, logits, bias, ws):
    moe.route(c, x, p["Wg"], p["bg"], b, logits=logits)
    moe.route_scores(s, logits, bias, b["idx"], b["w"], b["counts"], b["balance_loss"], ws)
    moe.dispatch(c, b["idx"], x, b)
    moe.expert_ffn(c, b["Xp"], b["offsets"], p["W1"], p["b1"], p["W2"], p["b2"], b)
    moe.combine(c, b["Yp"], b["slot_row"], b["w"], b["y"])


CASES = [
    # T, d, E, k, d_ff, dtype, kind, renorm, groups, kept, top, capacity
    (300, 64, 8, 2, 96, "f32", "softmax", True, 1, 1, 1, None),
    (300, 64, 8, 3, 96, "f32", "softmax", False, 1, 1, 1, 1.0),
    (301, 64, 40, 4, 64, "f32", "sigmoid", True, 8, 3, 2, 1.0),
    (123, 37, 10, 3, 45, "f32", "softmax", False, 2, 1, 1, None),          # odd rows
    (123, 37, 10, 3, 45, "f32", "sigmoid", False, 1, 1, 1, 1.25),
    (500, 128, 16, 4, 128, "bf16", "sigmoid", True, 4, 2, 2, 1.0),
    (500, 128, 16, 4, 128, "bf16", "softmax", False, 1, 1, 1, None),
    (700, 128, 64, 8, 128, "bf16", "sigmoid", True, 8, 4, 2, None),        # gate contractions on tensor cores
    (700, 128, 64, 8, 128, "bf16", "softmax", False, 1, 1, 1, 1.0),
    (400, 70, 12, 2, 33, "bf16", "softmax", False, 1, 1, 1, None),
    (1, 64, 8, 2, 64, "bf16", "sigmoid", True, 1, 1, 1, None),
    (2200, 128, 4, 2, 128, "bf16", "sigmoid", True, 1, 1, 1, None),        # expert products on CTA pairs
]


@pytest.mark.parametrize("T,d,E,k,f,dtype,kind,renorm,groups,kept,top,cap", CASES)
def test_layer(T, d, E, k, f, dtype, kind, renorm, groups, kept, top, cap, moe_lib, cuda_device):
    moe = moe_lib
    p, x, dy, bias = make(T, d, E, f, dtype)
    gate = (kind, renorm, 2.5, 0.7)
    c = moe.make_config(T, d, E, k, f, capacity_factor=cap, has_gate_bias=True, dtype=dtype)
    s = moe.make_score_config(T, E, k, score=kind, groups=groups, groups_kept=kept, group_top=top, renormalise=renorm,
                              scale=2.5, temperature=0.7)
    dev = {n: t.cuda() for n, t in p.items()}
    xd, dyd = x.cuda(), dy.cuda()
    b = moe.alloc_buffers(c)
    logits, dlogits = (torch.full((T, E), float("nan"), device="cuda") for _ in range(2))
    ws = torch.empty(moe.route_scores_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    forward(moe, c, s, dev, xd, b, logits, bias.cuda(), ws)
    moe.backward_scores(c, s, logits, dlogits, dyd, xd, dev["Wg"], dev["W1"], dev["W2"], b)
    moe.get_error()

    idx, kept_slots = b["idx"].long().cpu(), b["slot_row"].cpu() >= 0
    leaves = {n: t.double().requires_grad_(True) for n, t in p.items()}
    x64 = x.double().requires_grad_(True)
    y, z, w = layer64(x64, leaves, idx, kept_slots, gate)
    z.retain_grad()
    w.retain_grad()
    loss = (y * dy.double()).sum()
    loss.backward()
    tol = P.TOL[dtype]
    P.assert_close("y", P.f64(b["y"]), y.detach().numpy(), tol)
    P.assert_close("w", P.f64(b["w"]), w.detach().numpy(), tol)
    P.assert_close("dlogits", P.f64(dlogits), z.grad.numpy(), tol)
    for name, got, ref in (("dx", b["dx"], x64), ("dWg", b["dWg"], leaves["Wg"]), ("dbg", b["dbg"], leaves["bg"]),
                           ("dW1", b["dW1"], leaves["W1"]), ("db1", b["db1"], leaves["b1"]),
                           ("dW2", b["dW2"], leaves["W2"]), ("db2", b["db2"], leaves["b2"])):
        P.assert_close(name, P.f64(got), ref.grad.numpy(), tol)
    # the reported loss as the layer's own tests judge it: against the size of the sum's terms
    scale = float((y.detach() * dy.double()).norm())
    aux = 0.01 * float(b["balance_loss"])
    assert abs(float(b["loss"]) - aux - float(loss.detach())) <= tol * max(scale, abs(float(loss.detach()))) + 1e-6 * aux


def test_backward_of_the_plain_layer_is_what_it_was(moe_lib, cuda_device):
    """Renormalised softmax over all experts without bias or groups is the layer's own softmax over the k:
    both backward calls give the same gradients, to their roundings."""
    moe = moe_lib
    T, d, E, k, f = 400, 64, 16, 4, 64
    p, x, dy, _ = make(T, d, E, f, "f32", seed=5)
    dev = {n: t.cuda() for n, t in p.items()}
    c = moe.make_config(T, d, E, k, f, has_gate_bias=True, dtype="f32", temperature=0.7)
    s = moe.make_score_config(T, E, k, temperature=0.7)
    a, b = moe.alloc_buffers(c), moe.alloc_buffers(c)
    xd, dyd = x.cuda(), dy.cuda()
    moe.forward_backward(c, dev, xd, dyd, a)
    logits, dlogits = torch.empty(T, E, device="cuda"), torch.empty(T, E, device="cuda")
    forward(moe, c, s, dev, xd, b, logits, None, torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    moe.backward_scores(c, s, logits, dlogits, dyd, xd, dev["Wg"], dev["W1"], dev["W2"], b)
    moe.get_error()
    assert torch.equal(a["idx"], b["idx"]) and torch.equal(a["counts"], b["counts"])
    for n in ("w", "y", "dx", "dWg", "dbg", "dW1", "db1", "dW2", "db2", "loss"):
        P.assert_close(n, P.f64(b[n]), P.f64(a[n]), 1e-4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty_batch(dtype, moe_lib, cuda_device):
    moe = moe_lib
    p, x, dy, bias = make(0, 64, 8, 64, dtype)
    dev = {n: t.cuda() for n, t in p.items()}
    c = moe.make_config(0, 64, 8, 2, 64, has_gate_bias=True, dtype=dtype)
    s = moe.make_score_config(0, 8, 2, renormalise=False)
    b = moe.alloc_buffers(c)
    z = torch.empty(0, 8, device="cuda")
    for key in ("dWg", "dW1", "db1", "dW2", "db2", "loss"):
        b[key].fill_(7.0)
    forward(moe, c, s, dev, x.cuda(), b, z, bias.cuda(), torch.empty(1 << 16, dtype=torch.uint8, device="cuda"))
    moe.backward_scores(c, s, z, z.clone(), dy.cuda(), x.cuda(), dev["Wg"], dev["W1"], dev["W2"], b)
    moe.get_error()
    for key in ("dWg", "dW1", "db1", "dW2", "db2", "loss", "counts"):
        assert (b[key] == 0).all(), key


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_block(dtype, moe_lib, cuda_device):
    """x' = s + MoE(norm(s)) with s = x + r: all gradients of the block, and a Muon step on the experts,
    captured into one graph."""
    moe = moe_lib
    T, d, E, k, f = 384, 64, 16, 4, 96
    p, x, dy, bias = make(T, d, E, f, dtype, seed=7)
    g = torch.Generator().manual_seed(8)
    r = torch.randn(T, d, generator=g).to(DT[dtype])
    gain, shift = 1 + 0.1 * torch.randn(d, generator=g), 0.1 * torch.randn(d, generator=g)
    gate = ("sigmoid", True, 2.0, 1.0)
    c = moe.make_config(T, d, E, k, f, has_gate_bias=True, dtype=dtype)
    s = moe.make_score_config(T, E, k, score="sigmoid", groups=4, groups_kept=2, group_top=2, scale=2.0)
    n = moe.make_norm_config(T, d, dtype=dtype)
    dev = {name: t.cuda() for name, t in p.items()}
    start = {name: dev[name].clone() for name in ("W1", "W2")}
    xd, rd, dyd, gd, sd, bd = (t.cuda() for t in (x, r, dy, gain, shift, bias))
    total, normed, dn, dx = (torch.empty_like(xd) for _ in range(4))
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dgain, dshift = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    logits, dlogits = torch.empty(T, E, device="cuda"), torch.empty(T, E, device="cuda")
    b = moe.alloc_buffers(c)
    ws, wn = (torch.empty(q, dtype=torch.uint8, device="cuda")
              for q in (moe.route_scores_workspace_bytes(s), moe.norm_workspace_bytes(n)))
    opt = moe.Muon([dict(p=dev[w], g=b["d" + w]) for w in ("W1", "W2")], lr=0.01)

    def step():
        moe.layer_norm(n, xd, gd, sd, normed, residual=rd, total=total, mean=mean, rstd=rstd)
        forward(moe, c, s, dev, normed, b, logits, bd, ws)
        moe.backward_scores(c, s, logits, dlogits, dyd, normed, dev["Wg"], dev["W1"], dev["W2"], b, want_loss=False)
        moe.layer_norm_backward(n, b["dx"], total, gd, mean, rstd, dx, dgain, dshift, wn, dtotal=dyd)
        opt.step()

    def reset():
        for name, t in start.items():
            dev[name].copy_(t)
        for t in opt.tensors:
            t["m"].zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    eager = {name: b[name].clone() for name in ("dx", "dWg", "dW1", "dW2")}
    eager.update(dx_all=dx.clone(), dgain=dgain.clone(), W1=dev["W1"].clone(), W2=dev["W2"].clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    reset()
    graph.replay()
    torch.cuda.synchronize()
    moe.get_error()
    for name, t in eager.items():
        now = dx if name == "dx_all" else dgain if name == "dgain" else dev[name] if name in start else b[name]
        assert torch.equal(now, t), name

    leaves = {name: t.double().requires_grad_(True) for name, t in p.items()}
    x64, g64, s64 = (t.double().requires_grad_(True) for t in (x, gain, shift))
    tot = x64 + r.double()
    h = torch.nn.functional.layer_norm(tot, (d,), g64, s64, 1e-5)
    y, _, _ = layer64(h, leaves, b["idx"].long().cpu(), b["slot_row"].cpu() >= 0, gate)
    ((tot + y) * dy.double()).sum().backward()
    tol = P.TOL[dtype]
    P.assert_close("y", P.f64(b["y"]), y.detach().numpy(), tol)
    for name, got, ref in (("dx", dx, x64), ("dgain", dgain, g64), ("dshift", dshift, s64), ("dWg", b["dWg"], leaves["Wg"]),
                           ("dW1", b["dW1"], leaves["W1"]), ("dW2", b["dW2"], leaves["W2"])):
        P.assert_close(name, P.f64(got), ref.grad.numpy(), tol)
    # the step moves every expert's matrix by lr * scale times a matrix of singular values near one
    for name in start:
        moved = (start[name].double() - dev[name].double()) / (0.01 * 0.2 * max(d, f) ** 0.5)
        used = b["counts"].cpu() > 0
        top = torch.linalg.svdvals(moved.cpu())[used][:, 0]
        assert float(top.min()) > 0.6 and float(top.max()) < 1.3
