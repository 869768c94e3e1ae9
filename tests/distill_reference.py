"""Distillation from a teacher's top logits in 64 bits, from its definition, and the
error bounds the GPU tests hold the kernels to."""
import math

import torch

F64 = torch.float64


def teacher(ids, logits, V, temperature, teacher_lse=None):
    """(used mask, log q with 0 in empty slots, q) of the [N, K] lists."""
    a = logits.to(F64) / temperature
    used = (ids >= 0) & (ids < V) & (a != -math.inf)
    a = torch.where(used, a, -math.inf)
    if teacher_lse is None:
        norm = torch.logsumexp(a, 1) if a.size(1) else torch.zeros(a.size(0), dtype=F64)
    else:
        norm = teacher_lse.to(F64)
    logq = torch.where(used, a - norm[:, None], 0.0)
    return used, logq, torch.where(used, logq.exp(), 0.0)


def distill(hidden, weight, ids, logits, bias=None, temperature=1.0, teacher_lse=None):
    """(loss, lse) in 64 bits on the CPU."""
    z = hidden.to(F64) @ weight.to(F64).T
    if bias is not None:
        z = z + bias.to(F64)
    z = z / temperature
    lse = torch.logsumexp(z, 1)
    used, logq, q = teacher(ids, logits, weight.size(0), temperature, teacher_lse)
    zk = z.gather(1, torch.where(used, ids, 0))
    terms = torch.where(used, q * (logq - zk + lse[:, None]), 0.0)
    return temperature ** 2 * terms.sum(1), lse


def grad_logits(hidden, weight, ids, logits, grad, bias=None, temperature=1.0, teacher_lse=None):
    """dL/dz [N, V] for the upstream gradient grad [N]."""
    V = weight.size(0)
    z = hidden.to(F64) @ weight.to(F64).T
    if bias is not None:
        z = z + bias.to(F64)
    p = torch.softmax(z / temperature, 1)
    used, _, q = teacher(ids, logits, V, temperature, teacher_lse)
    G = p * q.sum(1, keepdim=True)
    for k in range(ids.size(1)):
        G.scatter_add_(1, torch.where(used[:, k], ids[:, k], 0)[:, None], -q[:, k:k + 1])
    return G * (grad.to(F64) * temperature)[:, None]


def logit_error(hidden, weight, bias=None):
    """A bound on |z - z exact| per row: H products summed in FP32 (H 2^-24 sum|h w|, the textbook
    bound) and the bias added once."""
    terms = hidden.to(F64).abs() @ weight.to(F64).abs().T
    if bias is not None:
        terms = terms + bias.to(F64).abs()
    return (hidden.size(1) + 2) * 2.0 ** -24 * terms.amax(1)


def bounds(hidden, weight, ids, logits, bias=None, temperature=1.0, teacher_lse=None):
    """(loss bound, lse bound, relative bound on p) per row.

    lse moves by at most the largest logit error over T, plus a few FP32 roundings of
    values up to |z|/T + |lse| (exponents carry them through 2^x, which the hardware
    evaluates to 2^-22).  The loss is T^2 sum q (log q - z/T + lse): q times both errors.
    """
    z = hidden.to(F64) @ weight.to(F64).T
    if bias is not None:
        z = z + bias.to(F64)
    z = z / temperature
    lse = torch.logsumexp(z, 1)
    dz = logit_error(hidden, weight, bias) / temperature
    size = z.abs().amax(1) + lse.abs() + 1
    dlse = dz + 2.0 ** -20 * size
    used, logq, q = teacher(ids, logits, weight.size(0), temperature, teacher_lse)
    size = size + (logits.to(F64) / temperature).masked_fill(~used, 0.0).abs().sum(1) / \
        used.sum(1).clamp(min=1) + logq.abs().amax(1) if ids.size(1) else size
    dloss = temperature ** 2 * (q.sum(1) + 1e-30) * (dz + dlse + 2.0 ** -19 * size)
    return dloss, dlse, 2 * (dz + dlse) + 2.0 ** -19 * size
