"""Training a small policy end to end through the library: tokens to a table's rows (embedding), a
gated feed-forward block with a residual, and the log-probability of the next token under a head that
is the same table (linear_logp), forward and backward.

Every product's sums have a fixed order and the table's gradient adds its rows in a fixed order, so two
runs give the same bits.  --checkpoint says what waits for the backward (see gated_linear_trainable);
"int8" holds the block's activations in 8 bits.

    python examples/tied_policy_training.py [--steps N] [--checkpoint fp32|int8|again]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import deterministic_invariant_gemm_linear_gb300 as rlk  # noqa: E402


def logp(tokens, targets, table, w_in, w_out, checkpoint=None):
    """log p(target | token) for each position; the three weights are bf16."""
    x = rlk.embedding_trainable(tokens, table)
    h = rlk.gated_linear_trainable(x, w_in, "silu", checkpoint=checkpoint)
    y = rlk.det_linear_trainable(h, w_out, checkpoint="int8" if checkpoint == "int8" else None)
    return rlk.linear_logp_trainable(x + y, table, targets)[0]


def start(hidden=256, inner=700, vocab=5000, seed=0):
    """FP32 master weights: the table, the block's two projections, its way back."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(vocab, hidden, device="cuda", generator=g).mul_(0.5),
            torch.randn(2 * inner, hidden, device="cuda", generator=g).div_(math.sqrt(hidden)),
            torch.randn(hidden, inner, device="cuda", generator=g).div_(math.sqrt(inner))]


def gradients(tokens, targets, master, checkpoint=None):
    """Loss (minus the mean log-probability) and its gradients of the bf16 weights."""
    weights = [m.bfloat16().requires_grad_() for m in master]
    loss = -logp(tokens, targets, *weights, checkpoint=checkpoint).mean()
    return loss.detach(), torch.autograd.grad(loss, weights)


def train(steps=20, batch=8, length=128, rate=0.5, checkpoint=None, seed=0, **sizes):
    """Runs the steps on a fixed synthetic text; returns (losses, master weights)."""
    master = start(seed=seed, **sizes)
    vocab = master[0].size(0)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    # the next token is a function of this one, commoner tokens first
    tokens = torch.rand(batch, length, device="cuda", generator=g, dtype=torch.float64)
    tokens = (tokens * math.log(vocab)).exp().long().clamp_(1, vocab) - 1
    targets = (tokens * 31 + 7) % vocab
    losses = []
    for step in range(steps):
        loss, grads = gradients(tokens, targets, master, checkpoint)
        for m, grad in zip(master, grads):
            m -= rate * grad.float()
        losses.append(loss.item())
        print(f"step {step:3d}  loss {losses[-1]:.4f}")
    return losses, master


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=20)
    parser.add_argument("--checkpoint", choices=["fp32", "int8", "again"])
    args = parser.parse_args()
    train(steps=args.steps, checkpoint=args.checkpoint)
