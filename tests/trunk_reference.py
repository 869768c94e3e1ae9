"""64-bit definitions of the trunk's operators (embedding, 8-bit blocks, gated block), written out
with elementary torch operations on float64 tensors, on whichever device the inputs are."""
import math

import torch

GROUP, BLOCK = 64, 32


# ------------------------------------------------------------------ embedding
def embedding(ids, weight, scale):
    known = (ids >= 0) & (ids < weight.size(0))
    rows = weight.double()[torch.where(known, ids, 0)] * scale
    return torch.where(known[..., None], rows, 0.0)


def embedding_grad(ids, grad, V, scale):
    known = (ids >= 0) & (ids < V)
    out = torch.zeros(V, grad.size(-1), dtype=torch.float64, device=grad.device)
    return out.index_add_(0, ids[known], grad.double()[known]) * scale


def embedding_grad_fp32(ids, grad, V, scale):
    """The defined order, in FP32 on the CPU: an id's rows in ascending order, 64 at a time, then
    the groups' sums, then the scale."""
    out = torch.zeros(V, grad.size(-1))
    grad = grad.float().cpu()
    ids = ids.cpu()
    for v in ids[(ids >= 0) & (ids < V)].unique().tolist():
        rows = torch.nonzero(ids == v).flatten().tolist()
        total = torch.zeros(grad.size(-1))
        for g in range(0, len(rows), GROUP):
            part = torch.zeros(grad.size(-1))
            for r in rows[g:g + GROUP]:
                part = part + grad[r]
            total = part if len(rows) <= GROUP else total + part
        out[v] = total * torch.tensor(scale, dtype=torch.float32)
    return out


# ------------------------------------------------------------------ blocks of 8 bits
def power(n):
    """2^n as float64, n int64 in -1022 .. 1023 (built from its bits: exact on every device)."""
    return ((n + 1023) << 52).view(torch.float64)


def int8_blocks(x):
    """(values, exponents) as whole numbers [rows, blocks, 32] and [rows, blocks] of x [rows, cols]."""
    x = torch.nn.functional.pad(x.double(), (0, -x.size(1) % BLOCK)).unflatten(1, (-1, BLOCK))
    bad = ~torch.isfinite(x).all(2)
    most = torch.where(bad, 1.0, x.abs().amax(2))
    # floor(log2 most): frexp's mantissa is 1/2 .. 1
    e = (torch.frexp(most).exponent.to(torch.int64) - 1 + 121).clamp(min=1)
    e = torch.where(most == 0, 1, e)
    q = (torch.where(bad[..., None], 0.0, x) * power(127 - e)[..., None]).round()
    return (torch.where(bad[..., None], 0.0, q.clamp(-127, 127)).to(torch.int64),
            torch.where(bad, 255, e))


def int8_values(q, e, cols):
    """What the blocks stand for, [rows, cols]."""
    x = q.double() * power(e.to(torch.int64) - 127)[..., None]
    return torch.where((e == 255)[..., None], math.nan, x).flatten(1)[:, :cols]


# ------------------------------------------------------------------ the gated block
def argument(g, act):
    """a(g) of act(g) = g sigmoid(a(g)), and a'(g)."""
    if act == "silu":
        return g, torch.ones_like(g)
    c = 2 * math.sqrt(2 / math.pi)
    return c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g * g)


def activation(g, act):
    """act(g) and act'(g)."""
    a, da = argument(g, act)
    s = torch.sigmoid(a)
    return g * s, s + g * s * torch.sigmoid(-a) * da


def gated(x, w, act):
    f = w.size(0) // 2
    z = x.double() @ w.double().t()
    return activation(z[..., :f], act)[0] * z[..., f:]


def gated_grad_projections(d, g, u, act):
    """dL/d[g, u] for d = dL/dh."""
    value, slope = activation(g.double(), act)
    return torch.cat([d.double() * u.double() * slope, d.double() * value], -1)
