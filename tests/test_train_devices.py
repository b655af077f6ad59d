"""The training-step binding refuses tensors that are not all on one GPU, before anything is launched.
CPU only: no call here has a GPU tensor."""
import pytest
import torch

F, I, B = torch.float32, torch.int32, torch.bfloat16


def z(*shape, dtype=F):
    return torch.zeros(*shape, dtype=dtype)


def test_host_tensors_are_refused(moe_lib):
    moe = moe_lib
    c = moe.make_embed_config(4, 6, 8)
    ids, W, y = z(4, dtype=I), z(6, 8, dtype=B), z(4, 8, dtype=B)
    ws = z(moe.embed_workspace_bytes(c), dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        moe.embed(c, ids, W, y)
    with pytest.raises(ValueError, match="GPU"):
        moe.embed_backward(c, ids, y, W, ws)
    c = moe.make_policy_config(4, 6, kl_weight=0.1)
    ws = z(moe.policy_workspace_bytes(c), dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        moe.token_logp(c, z(4, 6, dtype=B), ids, z(4))
    with pytest.raises(ValueError, match="GPU"):
        moe.policy_loss(c, z(4, 6, dtype=B), ids, z(4), z(4), z(4), z(4), z(4), z(1), z(4, 6, dtype=B), ws)
    for bits in (8, 32):
        opt = moe.AdamW([dict(p=z(300), g=z(300), master=z(300))], bits=bits)   # may be made, as for a checkpoint
        with pytest.raises(ValueError, match="GPU"):
            opt.step()
        with pytest.raises(ValueError, match="GPU"):
            opt.step(lr=z(1), grad_scale=z(1))


class On:
    """What the check sees of a tensor on a given device (-1: the host)."""

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device


@pytest.mark.parametrize("devices", [(0, -1), (-1, 0), (0, 1), (0, 0, None, 1), (-1, None), (-1, -1)])
def test_mixed_devices_are_refused(devices, moe_lib):
    from token_routing_gb300 import train
    with pytest.raises(ValueError, match="GPU"):
        train._one_gpu(*(None if d is None else On(d) for d in devices))


def test_one_gpu_is_taken(moe_lib):
    from token_routing_gb300 import train
    assert train._one_gpu(On(0), None, On(0)) == 0 and train._one_gpu(On(1), On(1)) == 1


@pytest.mark.parametrize("what", ["p", "g", "master", "m", "v", "m_scale", "v_scale", "state", "lr", "grad_scale"])
def test_adamw_looks_at_every_array(what, moe_lib, monkeypatch):
    """Every array that a step hands over is looked at: one alone on another device is refused."""
    from token_routing_gb300 import train
    opt = moe_lib.AdamW([dict(p=z(300), g=z(300)), dict(p=z(30), g=z(30), master=z(30))], bits=8)
    given = dict(lr=z(1), grad_scale=z(1))
    odd = opt.state if what == "state" else given.get(what, opt.tensors[1].get(what))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0 if t is not odd else -1)
    monkeypatch.setattr(train.L, "load", lambda: pytest.fail("launched"))
    with pytest.raises(ValueError, match="GPU"):
        opt.step(**given)
