"""A policy trained with the framework's operators and its optimizer step.

A contextual bandit: each context has one action that pays 1.  The policy is a
small pre-norm network; a training step runs

    layer norm -> 8-bit linear -> ReLU -> 8-bit linear
    -> residual + dropout + layer norm (one kernel) -> 8-bit linear -> logits
    -> clipped policy loss with a KL penalty to the first policy, and its gradient
    -> the same backwards: float32 gradients of the three weight matrices
    -> RotatedAdam on those, plain descent on the norms' vectors

    python examples/policy_step.py [--steps 200]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from matrix_optimizer_step_rot_gb300 import binding as B  # noqa: E402
from matrix_optimizer_step_rot_gb300 import operators as ops  # noqa: E402
from matrix_optimizer_step_rot_gb300.optimizer import RotatedAdam  # noqa: E402

CONTEXTS, ACTIONS, WIDTH, HIDDEN, DROP = 32, 32, 128, 256, 0.05


class Policy:
    def __init__(self, seed: int):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(*shape, generator=g, device="cuda") * std

        self.embed = normal(CONTEXTS, WIDTH, std=1.0).bfloat16()
        # the optimizer's matrices: up, down, out
        self.w = [normal(HIDDEN, WIDTH, std=WIDTH ** -0.5), normal(WIDTH, HIDDEN, std=HIDDEN ** -0.5),
                  normal(ACTIONS, WIDTH, std=0.1 * WIDTH ** -0.5)]
        self.norms = [torch.ones(WIDTH, device="cuda"), torch.zeros(WIDTH, device="cuda"),
                      torch.ones(WIDTH, device="cuda"), torch.zeros(WIDTH, device="cuda")]
        self.quantize()

    def quantize(self) -> None:
        """The weights in 8 bits, both orientations, after they have changed."""
        self.q, self.qt = zip(*(ops.fp8_quantize(w, block_rows=128, transposed=True) for w in self.w))

    def forward(self, contexts: torch.Tensor, p: float = 0.0, seed: int = 0, offset: int = 0):
        """(logits, what the backward pass needs)."""
        g1, b1, g2, b2 = self.norms
        y1, h1, m1, r1 = ops.layer_norm(self.embed[contexts], g1, b1)
        u = ops.fp8_linear(y1, self.q[0])
        a = torch.relu(u)
        v = ops.fp8_linear(a, self.q[1])
        y2, h2, m2, r2 = ops.layer_norm(v, g2, b2, residual=h1, p=p, seed=seed, offset=offset)
        return ops.fp8_linear(y2, self.q[2]), (y1, h1, m1, r1, u, a, y2, h2, m2, r2, p, seed, offset)

    def backward(self, dlogits: torch.Tensor, saved):
        """(float32 gradients of the matrices, of the norms' vectors)."""
        y1, h1, m1, r1, u, a, y2, h2, m2, r2, p, seed, offset = saved
        g1, _, g2, _ = self.norms
        dy2, dw_out = ops.fp8_linear_backward(dlogits, y2, self.qt[2])
        dv, dh1, dg2, db2 = ops.layer_norm_backward(dy2, h2, m2, r2, g2, p=p, seed=seed, offset=offset)
        da, dw_down = ops.fp8_linear_backward(dv, a, self.qt[1])
        dy1, dw_up = ops.fp8_linear_backward(torch.where(u > 0, da, 0), y1, self.qt[0])
        _, _, dg1, db1 = ops.layer_norm_backward(dy1, h1, m1, r1, g1, dh=dh1)
        return [dw_up, dw_down, dw_out], [dg1, db1, dg2, db2]


def train(steps: int = 200, tokens: int = 1024, seed: int = 0, say=print):
    """Mean reward of every step."""
    policy, first = Policy(seed), Policy(seed)
    opt = RotatedAdam([tuple(w.shape) for w in policy.w], 64 << 20, lr=2e-3,
                      precision=B.ROT_PREC_3XF16)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    paying = torch.randperm(CONTEXTS, generator=g, device="cuda") % ACTIONS
    weights = torch.full((tokens,), 1.0 / tokens, device="cuda")
    rewards = []
    for step in range(1, steps + 1):
        contexts = torch.randint(CONTEXTS, (tokens,), generator=g, device="cuda")
        logits, _ = policy.forward(contexts)
        actions = torch.multinomial(torch.softmax(logits.float(), 1), 1, generator=g)[:, 0]
        reward = (actions == paying[contexts]).float()
        rewards.append(reward.mean())
        advantages = reward - reward.mean()
        advantages = advantages / (advantages.std() + 1e-3)
        old = ops.token_logprobs(logits, actions)
        ref = ops.token_logprobs(first.forward(contexts)[0], actions)
        for again in range(2):  # two updates on the same samples: the second one's ratios are clipped
            logits, saved = policy.forward(contexts, DROP, seed, 2 * step + again)
            loss, _, d = ops.policy_loss(logits, actions, old, advantages, weights, ref_logp=ref,
                                         kl_coef=0.002, out=logits)
            dw, dn = policy.backward(d, saved)
            opt.step(policy.w, dw, refresh=(2 * step + again) % 10 == 0)
            for v, dv in zip(policy.norms, dn):
                v.sub_(dv, alpha=0.02)
            policy.quantize()
        if say and (step == 1 or step % 20 == 0):
            say(f"step {step:4d}  reward {rewards[-1].item():.3f}  loss {loss.item():+.4f}")
    if opt.status() != B.ROT_OK or ops.status() != B.ROT_OK:
        raise RuntimeError("a device status word is set")
    return torch.stack(rewards).tolist()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    train(ap.parse_args().steps)
