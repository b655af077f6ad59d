"""The binding's check of a workspace is for the GPU that the tensors are on: a GPU with more SMs wants a larger one.
CPU only: GPUs and the library are stand-ins."""
import contextlib

import pytest
import torch

F, I, B = torch.float32, torch.int32, torch.bfloat16


class Machine:
    """GPU i has 100 (i + 1) SMs; workspaces are 4 bytes to each."""

    def __init__(self, monkeypatch, train):
        self.current, self.asked, self.launched, self.on = 0, 0, [], 0
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.current, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda gpu: 0, raising=False)
        monkeypatch.setattr(torch.cuda, "device", self.device)
        monkeypatch.setattr(torch.Tensor, "get_device", lambda t: self.on)
        monkeypatch.setattr(train.L, "load", lambda: self)
        monkeypatch.setattr(train, "_CALLS", {})

    @contextlib.contextmanager
    def device(self, gpu):
        was, self.current = self.current, gpu
        yield
        self.current = was

    def _size(self, cfg):
        self.asked += 1
        return 400 * (self.current + 1)

    moe_route_scores_workspace_bytes = moe_norm_workspace_bytes = _size

    def _launch(self, *args):
        self.launched.append(self.current)
        return 0

    moe_route_scores = moe_layer_norm_backward = _launch


@pytest.fixture
def machine(moe_lib, monkeypatch):
    from token_routing_gb300 import train
    return Machine(monkeypatch, train)


def z(*shape, dtype=F):
    return torch.zeros(*shape, dtype=dtype)


def calls(moe):
    c = moe.make_score_config(4, 8, 2)
    yield lambda ws: moe.route_scores(c, z(4, 8), None, z(4, 2, dtype=I), z(4, 2), counts=z(8, dtype=I), ws=ws)
    n = moe.make_norm_config(4, 8)
    x = z(4, 8, dtype=B)
    yield lambda ws: moe.layer_norm_backward(n, x, x, None, z(4), z(4), x, z(8), None, ws)


def test_a_size_of_another_gpu_is_not_taken(moe_lib, machine):
    for call in calls(moe_lib):
        machine.on = 0
        call(z(100))                                   # 400 bytes: enough on GPU 0
        machine.on = 1
        with pytest.raises(ValueError, match="800"):   # the same configuration on a GPU with more SMs
            call(z(100))
        call(z(200))
        machine.on = 0
        call(z(100))
    assert machine.launched == [0, 1, 0] * 2 and machine.current == 0


def test_the_current_gpu_need_not_be_theirs(moe_lib, machine):
    for call in calls(moe_lib):
        machine.current, machine.on = 1, 0             # the first question is asked while GPU 1 is current
        call(z(100))
        machine.on = 2
        with pytest.raises(ValueError, match="1200"):
            call(z(200))


def test_asked_once(moe_lib, machine):
    for call in calls(moe_lib):
        before = machine.asked
        for _ in range(3):
            call(z(100))
        assert machine.asked == before + 1
