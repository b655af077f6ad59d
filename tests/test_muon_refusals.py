"""A step of Muon that one of its tensors is refused for moves none of them. CPU only: the library is a stand-in."""
import pytest
import torch


def z(*shape):
    return torch.zeros(*shape)


def odd(*shape):
    """A contiguous tensor that starts 4 bytes behind a 16-byte boundary."""
    n = 1
    for s in shape:
        n *= s
    base = torch.zeros(n + 8)
    skip = (-base.data_ptr() // 4) % 4 + 1
    return base[skip:skip + n].view(*shape)


@pytest.mark.parametrize("what", ["p", "g", "m", "master"])
def test_nothing_moves_when_a_later_tensor_is_misaligned(what, moe_lib, monkeypatch):
    from token_routing_gb300 import train
    last = dict(p=z(8, 4), g=z(8, 4), m=z(8, 4), master=z(8, 4))
    last[what] = odd(8, 4)
    assert last[what].data_ptr() % 16 == 4 and last[what].is_contiguous()
    opt = moe_lib.Muon([dict(p=z(8, 4), g=z(8, 4)), last])
    launched = []
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(train, "_launch", lambda *a: launched.append(a))
    for _ in range(2):
        with pytest.raises(ValueError, match="16-byte"):
            opt.step()
    assert launched == []
    good = moe_lib.Muon([dict(p=z(8, 4), g=z(8, 4)), dict(p=z(3, 8, 4), g=z(3, 8, 4))])
    good.step()
    assert len(launched) == 2
