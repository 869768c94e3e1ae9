"""On-policy distillation of a linear policy head, every step through the library.

Each step draws one token a row from the student's own distribution (det_linear logits,
sample_logits), scores the drawn tokens under the unfiltered policy (linear_logp), asks the
teacher for its top logits at the same rows, and takes a gradient step on the distillation
loss (linear_distill_trainable).  The features stand for a trunk's hidden states.

    python examples/on_policy_distillation.py [--steps N]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import deterministic_invariant_gemm_linear_gb300 as rlk  # noqa: E402


def train(steps=20, rows=512, hidden=512, vocab=8000, slots=32, temperature=1.0, rate=20.0, seed=0):
    """Runs the steps; returns (losses, tokens of the last step, final weight)."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    features = torch.randn(rows, hidden, device=dev, generator=g).bfloat16()
    teacher = (torch.randn(vocab, hidden, device=dev, generator=g) * (3 / math.sqrt(hidden))).bfloat16()
    master = torch.randn(vocab, hidden, device=dev, generator=g) / math.sqrt(hidden)   # FP32 weights
    losses = []
    for step in range(steps):
        student = master.bfloat16().requires_grad_()
        # rollout: the student draws, with one given uniform number a row
        logits = rlk.det_linear(features, student.detach(), out_dtype=torch.float32)
        uniform = torch.rand(rows, device=dev, dtype=torch.float64, generator=g)
        token, drawn_logp = rlk.sample_logits(logits, uniform, temperature=0.9, top_k=100, top_p=0.95)
        policy_logp, _ = rlk.linear_logp(features, student.detach(), token)
        # the teacher's top logits at the visited rows
        best = rlk.det_linear(features, teacher, out_dtype=torch.float32).topk(slots, dim=1)
        loss, _ = rlk.linear_distill_trainable(features, student, best.indices, best.values,
                                               temperature=temperature)
        loss.mean().backward()
        master -= rate * student.grad.float()
        losses.append(loss.mean().item())
        print(f"step {step:3d}  loss {losses[-1]:.4f}  mean log-probability of the drawn tokens "
              f"{policy_logp.mean().item():.3f} (among those kept {drawn_logp.mean().item():.3f})")
    return losses, token, master


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=20)
    train(steps=parser.parse_args().steps)
