"""A policy trained by clipped policy steps: token embedding, the MoE layer, a head tied to the
embedding table, the policy loss with a KL term to the starting policy, all gradients, AdamW.

The task needs no data: the context is one token, an answer earns a reward when it has the context's
remainder modulo 8. Each round samples answers with the current policy, keeps their
log-probabilities (token_logp) and takes a few updates on them; an update is captured into a CUDA
graph once and replayed.

    python examples/policy_step.py [--rounds 60] [--bits 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import token_routing_gb300 as moe  # noqa: E402


class Policy:
    """Answers ~ softmax((x + MoE(x)) W^T / tau) with x = tau W[ids], tau = sqrt(d); every buffer of a step
    is made here."""

    def __init__(self, T=2048, V=512, d=256, E=8, k=2, d_ff=512, kl_weight=0.01, lr=3e-3, bits=32, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        f32 = dict(dtype=torch.float32, device="cuda")

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5).bfloat16()

        self.V, self.tau = V, d ** 0.5
        self.layer = moe.make_config(T, d, E, k, d_ff)
        self.table = moe.make_embed_config(T, V, d, scale=self.tau, grad_dtype="f32", accumulate=True)
        self.loss_cfg = moe.make_policy_config(T, V, temperature=self.tau, kl_weight=kl_weight)
        self.p = dict(W=weight(V, d), Wg=weight(E, d), bg=None, W1=weight(E, d_ff, d), b1=torch.zeros(E, d_ff, **bf),
                      W2=weight(E, d, d_ff), b2=torch.zeros(E, d, **bf))
        self.b = moe.alloc_buffers(self.layer, backward=True)
        self.ids, self.answer = (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(2))
        self.advantage, self.old, self.ref, self.logp = (torch.zeros(T, **f32) for _ in range(4))
        self.weight = torch.full((T,), 1.0 / T, **f32)
        self.x, self.h, self.dh = (torch.empty(T, d, **bf) for _ in range(3))
        self.logits = torch.empty(T, V, **bf)
        self.loss = torch.zeros(1, **f32)
        self.dW = torch.zeros(V, d, **f32)
        self.ws_embed = torch.empty(moe.embed_workspace_bytes(self.table), dtype=torch.uint8, device="cuda")
        self.ws_loss = torch.empty(moe.policy_workspace_bytes(self.loss_cfg), dtype=torch.uint8, device="cuda")
        grads = dict(W=self.dW, Wg=self.b["dWg"], W1=self.b["dW1"], b1=self.b["db1"], W2=self.b["dW2"], b2=self.b["db2"])
        self.opt = moe.AdamW([dict(p=self.p[n].view(-1), g=grads[n].view(-1), master=self.p[n].float().view(-1))
                              for n in grads], lr=lr, beta2=0.99, bits=bits)
        self.start = {n: None if w is None else w.clone() for n, w in self.p.items()}

    def forward(self, p=None):
        """self.logits of self.ids under the weights p (default: the current ones)."""
        p = p or self.p
        moe.embed(self.table, self.ids, p["W"], self.x)
        moe.forward(self.layer, p, self.x, self.b)
        torch.add(self.x, self.b["y"], out=self.h)
        torch.mm(self.h, p["W"].t(), out=self.logits)

    def update(self):
        """One step on (ids, answer, advantage, old, ref): loss, gradients, AdamW."""
        self.forward()
        # the gradient takes the logits' place
        moe.policy_loss(self.loss_cfg, self.logits, self.answer, self.advantage, self.old, self.ref, self.weight,
                        self.logp, self.loss, self.logits, self.ws_loss)
        self.dW.copy_(self.logits.t() @ self.h)                       # the head's part of the tied gradient
        torch.mm(self.logits, self.p["W"], out=self.dh)
        moe.backward(self.layer, self.dh, self.x, self.p["Wg"], self.p["W1"], self.p["W2"], self.b, want_dbg=False,
                     want_dw=False, want_loss=False)
        self.dh.add_(self.b["dx"])                                    # through the layer, and past it
        moe.embed_backward(self.table, self.ids, self.dh, self.dW, self.ws_embed)
        self.opt.step()

    def rollout(self, g):
        """Sample contexts and answers with the current policy; rewards' mean. Fills what update() takes."""
        T = self.ids.numel()
        self.ids.copy_(torch.randint(0, self.V, (T,), generator=g, device="cuda"))
        self.forward(self.start)
        reference = self.logits.clone()
        self.forward()
        probs = torch.softmax(self.logits.float() / self.tau, 1)
        self.answer.copy_(torch.multinomial(probs, 1, generator=g)[:, 0])
        moe.token_logp(self.loss_cfg, self.logits, self.answer, self.old)
        moe.token_logp(self.loss_cfg, reference, self.answer, self.ref)
        reward = (self.answer % 8 == self.ids % 8).float()
        self.advantage.copy_((reward - reward.mean()) / (reward.std() + 1e-6))
        return float(reward.mean())


def train(rounds=60, updates=2, seed=0, say=print, **sizes):
    """Mean reward of every round."""
    policy = Policy(seed=seed, **sizes)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    rewards, graph = [], None
    for r in range(rounds):
        rewards.append(policy.rollout(g))
        for _ in range(updates):
            if r == 0:
                policy.update()                       # eager: first calls resolve what a capture must not
            else:
                if graph is None:
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph):
                        policy.update()
                graph.replay()
        if say and (r % 10 == 9 or r == 0):
            say(f"round {r + 1}: mean reward {rewards[-1]:.3f}, loss {float(policy.loss):+.4f}, "
                f"{policy.opt.steps_done()} steps")
    moe.get_error()
    return rewards, policy


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--rounds", type=int, default=60)
    ap.add_argument("--bits", type=int, default=32, choices=(8, 32))
    a = ap.parse_args()
    train(rounds=a.rounds, bits=a.bits)
