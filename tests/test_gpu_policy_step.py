"""The training-step calls together with the layer, as examples/policy_step.py runs them."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import train_oracle as O

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "policy_step.py")


@pytest.fixture(scope="module")
def example(moe_lib):
    spec = importlib.util.spec_from_file_location("policy_step", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("bits", [32, 8])
def test_policy_learns(bits, example, cuda_device):
    """An eighth of the answers is right at first; trained, most are. Graph replays count their steps."""
    rewards, policy = example.train(rounds=40, updates=2, say=None, bits=bits, T=1024, V=64, d=128, d_ff=256)
    assert abs(rewards[0] - 0.125) < 0.06 and np.mean(rewards[-5:]) > 0.5
    assert policy.opt.steps_done() == 80


def test_gradient_of_the_whole_step(example, moe_lib, cuda_device):
    """The loss along the tied table's and the head's gradient: a small step against it lowers the loss
    by its squared length (first order; bf16 forward passes, so the step is one that moves the logits
    visibly and the agreement is to a fifth)."""
    policy = example.Policy(T=512, V=64, d=128, E=4, d_ff=128, kl_weight=0.0, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    policy.rollout(g)
    policy.forward()
    moe = moe_lib
    moe.policy_loss(policy.loss_cfg, policy.logits, policy.answer, policy.advantage, policy.old, None, policy.weight,
                    policy.logp, policy.loss, None, policy.ws_loss)
    base = float(policy.loss)
    ref = O.policy(policy.logits.double().cpu().numpy(), policy.answer.cpu().numpy(), policy.advantage.double().cpu().numpy(),
                   policy.old.double().cpu().numpy(), None, policy.weight.double().cpu().numpy(), tau=np.float64(np.float32(policy.tau)))
    assert abs(base - ref["loss"]) < 1e-6
    master = policy.p["W"].float()
    policy.opt.step = lambda: None
    policy.update()
    dW = policy.dW.clone()
    step = 2e-2 / float(dW.norm())
    policy.p["W"].copy_(master - step * dW)
    policy.forward()
    moe.policy_loss(policy.loss_cfg, policy.logits, policy.answer, policy.advantage, policy.old, None, policy.weight,
                    policy.logp, policy.loss, None, policy.ws_loss)
    moved = float(((policy.p["W"].float() - master) * dW).sum())
    assert moved < 0 and abs(float(policy.loss) - base - moved) < 0.2 * abs(moved)
    moe.get_error()
