"""Measured cases of the operators of a network's trunk, with their plain forms.

``embed``        rows of an embedding table for given ids, scaled.
``embed_train``  the same and the table's gradient.
``gated``        the gated block of a feed-forward layer: two projections of the
                 same rows, the gate's activation and the product.
``gated_train``  the same and the gradients of its input and weight, with the
                 projections held in 32 bits, held in 8 bits (the input too) or
                 formed again.
``linear_train`` a linear layer whose input waits for the backward in 8 bits.
``pack``         activations to 8 bits and back.

8 bits: blocks of 32 columns of a row share a power of two, 2^(e - 127) with
e = max(1, floor(log2 max|x|) + 121), and hold whole numbers of -127 .. 127.

Where ``own`` is false ``run`` computes a case with elementary torch operations;
where it is true it calls the framework.
"""
import math

import torch

own = False

BF16_BYTES, FP32_BYTES, INT64_BYTES = 2, 4, 8
BLOCK = 32


# ------------------------------------------------------------------ the cases
def _embed(name, kind, rows, hidden, vocab, dtype="bf16", scale=1.0, padded=False):
    return {"name": name, "kind": kind, "rows": rows, "hidden": hidden, "vocab": vocab,
            "dtype": dtype, "scale": scale, "padded": padded}


def _gated(name, kind, rows, hidden, inner, act="silu", hold="", pitch=0):
    return {"name": name, "kind": kind, "rows": rows, "hidden": hidden, "inner": inner, "act": act,
            "hold": hold, "pitch": pitch}


def _linear(name, rows, hidden, inner):
    return {"name": name, "kind": "linear_train", "rows": rows, "hidden": hidden, "inner": inner}


def _pack(name, rows, hidden, dtype="bf16"):
    return {"name": name, "kind": "pack", "rows": rows, "hidden": hidden, "dtype": dtype}


def listed():
    return [
        # one token of one request enters the network: latency is all there is
        _embed("embed one token", "embed", 1, 4096, 151936),
        # a large micro-batch of prompts, scaled by the root of the width
        _embed("embed batch", "embed", 16384, 5120, 152064, scale=math.sqrt(5120)),
        # a short odd training batch at a small table, FP32 master weights
        _embed("embed train ragged", "embed_train", 255, 2048, 32003, "fp32", padded=True),
        # the gradient of a whole table from a large micro-batch, a tenth of it one id
        _embed("embed train batch", "embed_train", 16384, 4096, 151936, padded=True),
        # one token through the block: the weight is streamed once
        _gated("gated one token", "gated", 1, 4096, 16384),
        # a decode batch of a few rows at odd widths and an odd pitch
        _gated("gated 17 rows", "gated", 17, 2048, 5461, "gelu_tanh", pitch=2051),
        # a prompt's worth of rows: tensor cores
        _gated("gated batch", "gated", 4096, 4096, 16384),
        # training step of the smallest network: launches and latency
        _gated("gated train tiny", "gated_train", 64, 256, 1024, "gelu_tanh", "fp32"),
        # a short odd batch, everything that waits for the backward in 8 bits
        _gated("gated train ragged", "gated_train", 255, 2048, 5461, "silu", "int8"),
        # a micro-batch of a wide network
        _gated("gated train batch", "gated_train", 4096, 4096, 16384, "silu", "fp32"),
        # a linear layer that keeps its input in 8 bits
        _linear("linear train in 8 bits", 2048, 4096, 4096),
        # a layer's activations to 8 bits and back
        _pack("pack batch", 16384, 4096),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _unnamed(case):
    return {k: v for k, v in case.items() if k != "name"}


def draw(rng):
    kind = rng.choice(["embed", "embed_train", "gated", "gated_train", "gated_train", "linear_train",
                       "pack"])
    hidden = rng.choice([256, 512, 1000, 1024, 1537, 2048, 4096, 5120])
    if kind.startswith("embed"):
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        vocab = _log_int(rng, 1000, 151936 if hidden < 5120 and dtype == "bf16" else 60000)
        return _unnamed(_embed("", kind, _log_int(rng, 1, 16384), hidden, vocab, dtype,
                               rng.choice([1.0, math.sqrt(hidden), 0.125]), rng.random() < 0.5))
    if kind == "pack":
        return _unnamed(_pack("", _log_int(rng, 1, 16384), rng.randrange(32, 4097),
                              rng.choice(["bf16", "fp32"])))
    rows, hidden = _log_int(rng, 1, 4096), min(hidden, 4096)
    if kind == "linear_train":
        return _unnamed(_linear("", rows, hidden, _log_int(rng, 64, 4096)))
    pitch = rng.choice([0, 0, hidden + rng.randrange(1, 9)])
    hold = rng.choice(["fp32", "int8", "again"]) if kind == "gated_train" else ""
    return _unnamed(_gated("", kind, rows, hidden, _log_int(rng, 64, 16384),
                           rng.choice(["silu", "gelu_tanh"]), hold, pitch))


def work(case):
    n, h, kind = case["rows"], case["hidden"], case["kind"]
    if kind.startswith("embed"):
        size = FP32_BYTES if case["dtype"] == "fp32" else BF16_BYTES
        moved, flops = n * INT64_BYTES + 2 * n * h * size, n * h
        if kind == "embed_train":
            moved += n * h * size + case["vocab"] * h * size
            flops += n * h
        return {"bytes": moved, "flops": flops}
    if kind == "pack":
        size = FP32_BYTES if case["dtype"] == "fp32" else BF16_BYTES
        packed = n * h + n * -(-h // BLOCK)
        return {"bytes": n * h * (size + BF16_BYTES) + 2 * packed, "flops": 4 * n * h}
    f = case["inner"]
    if kind == "linear_train":
        moved = 2 * BF16_BYTES * (n * h + n * f + f * h)       # each tensor and its gradient
        return {"bytes": moved, "flops": 6 * n * h * f}
    moved = BF16_BYTES * (n * h + 2 * f * h + n * f)
    flops = 4 * n * h * f
    if kind == "gated_train":
        return {"bytes": 2 * moved, "flops": 3 * flops}
    return {"bytes": moved, "flops": flops}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _activations(rows, cols, g):
    # normed rows with a few columns that stand out, as a residual stream has
    x = torch.randn(rows, cols, device="cuda", generator=g)
    loud = torch.randint(cols, (max(1, cols // 128),), device="cuda", generator=g)
    x[:, loud] *= 6.0
    return x


def prepare(case, seed):
    g = _generator(seed)
    n, h, kind = case["rows"], case["hidden"], case["kind"]
    if kind.startswith("embed"):
        dtype = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        v = case["vocab"]
        weight = torch.randn(v, h, device="cuda", generator=g).to(dtype)
        # ids as text has them: the k-th commonest about 1/k as common as the first
        ids = torch.rand(n, device="cuda", generator=g, dtype=torch.float64).mul_(math.log(v)).exp_()
        ids = ids.floor_().to(torch.int64).clamp_(1, v) - 1
        ids = (ids * 7919 + 11) % v               # spread over the table
        if case["padded"]:                        # a tenth one id, a few that stand for nothing
            r = torch.rand(n, device="cuda", generator=g)
            ids = torch.where(r < 0.1, 0, torch.where(r > 0.97, -1, ids))
        s = {"kind": kind, "ids": ids, "weight": weight, "scale": case["scale"]}
        if kind == "embed_train":
            s["grad"] = torch.randn(n, h, device="cuda", generator=g).to(dtype)
        return s
    if kind == "pack":
        x = _activations(n, h, g)
        return {"kind": kind, "x": x if case["dtype"] == "fp32" else x.bfloat16()}
    f = case["inner"]
    x = _activations(n, case.get("pitch") or h, g).bfloat16()[:, :h]
    rows = f if kind == "linear_train" else 2 * f
    weight = torch.randn(rows, h, device="cuda", generator=g).mul_(1.0 / math.sqrt(h)).bfloat16()
    s = {"kind": kind, "x": x, "weight": weight, "act": case.get("act"), "hold": case.get("hold")}
    if kind != "gated":
        s["grad"] = torch.randn(n, f, device="cuda", generator=g).bfloat16()
    if kind == "linear_train":
        x.requires_grad_()
        weight.requires_grad_()
    return s


# ------------------------------------------------------------------ the plain forms
def _plain_embed(s):
    ids, weight, scale = s["ids"], s["weight"], s["scale"]
    v, h = weight.shape
    known = (ids >= 0) & (ids < v)
    at = torch.where(known, ids, 0)
    out = weight[at].float() * scale
    out = torch.where(known[:, None], out, 0.0).to(weight.dtype)
    if s["kind"] == "embed":
        return {"out": out}
    grad = torch.where(known[:, None], s["grad"].float() * scale, 0.0)
    table = torch.zeros(v, h, device="cuda").index_add_(0, at, grad)
    return {"out": out, "grad_weight": table.to(weight.dtype)}


def _blocks(x):
    """Whole numbers [rows, cols] and exponents [rows, blocks] of rows of FP32 numbers."""
    n, k = x.shape
    wide = torch.nn.functional.pad(x, (0, -k % BLOCK)).view(n, -1, BLOCK)
    e = (wide.abs().amax(2).view(torch.int32) >> 23) - 6
    e = e.clamp_(min=1)
    inverse = ((254 - e) << 23).view(torch.float32)
    q = (wide * inverse[:, :, None]).round_().clamp_(-127, 127)
    return q, e


def _through_8_bits(x):
    q, e = _blocks(x)
    return (q * (e << 23).view(torch.float32)[:, :, None]).view(x.size(0), -1)[:, :x.size(1)]


def _sigmoid(a):
    return 1.0 / (1.0 + torch.exp(-a))


TANH_SLOPE, TANH_CUBE = 2.0 * math.sqrt(2.0 / math.pi), 0.044715


def _gate(g, act):
    """The gate's activation g * sigmoid(a(g)) and its derivative."""
    if act == "silu":
        s = _sigmoid(g)
        return g * s, s + g * s * (1.0 - s)
    s = _sigmoid(TANH_SLOPE * (g + TANH_CUBE * g * g * g))
    return g * s, s + g * s * (1.0 - s) * TANH_SLOPE * (1.0 + 3.0 * TANH_CUBE * g * g)


def _plain_gated(s):
    x, w = s["x"].float(), s["weight"].float()
    f = w.size(0) // 2
    z = x @ w.t()
    value, slope = _gate(z[:, :f], s["act"])
    out = {"h": (value * z[:, f:]).bfloat16()}
    if s["kind"] == "gated":
        return out
    if s["hold"] == "int8":
        z = torch.cat([_through_8_bits(z[:, :f]), _through_8_bits(z[:, f:])], 1)
        x = _through_8_bits(x)
        value, slope = _gate(z[:, :f], s["act"])
    grad = s["grad"].float()
    dz = torch.cat([grad * z[:, f:] * slope, grad * value], 1)
    out["grad_x"] = (dz @ w).bfloat16()
    out["grad_weight"] = (dz.t() @ x).bfloat16()
    return out


def _plain_linear(s):
    x, w, grad = s["x"].detach().float(), s["weight"].detach().float(), s["grad"].float()
    return {"y": (x @ w.t()).bfloat16(), "grad_x": (grad @ w).bfloat16(),
            "grad_weight": (grad.t() @ _through_8_bits(x)).bfloat16()}


def _plain_pack(s):
    x = s["x"].float()
    n, k = x.shape
    q, e = _blocks(x)
    back = (q * (e << 23).view(torch.float32)[:, :, None]).view(n, -1)[:, :k]
    return {"values": q.view(n, -1)[:, :k].to(torch.int8), "exponents": e.to(torch.uint8),
            "back": back.bfloat16()}


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    kind = s["kind"]
    if not own:
        with torch.no_grad():
            if kind.startswith("embed"):
                return _plain_embed(s)
            return {"pack": _plain_pack, "linear_train": _plain_linear}.get(kind, _plain_gated)(s)
    import deterministic_invariant_gemm_linear_gb300 as rlk
    if kind.startswith("embed"):
        out = {"out": rlk.embedding(s["ids"], s["weight"], s["scale"])}
        if kind == "embed_train":
            out["grad_weight"] = rlk.embedding_backward(s["grad"], s["ids"], s["weight"].size(0),
                                                        s["scale"], s["weight"].dtype)
        return out
    if kind == "pack":
        values, exponents = rlk.pack_int8(s["x"])
        return {"values": values, "exponents": exponents, "back": rlk.unpack_int8(values, exponents)}
    x, w = s["x"], s["weight"]
    if kind == "gated":
        return {"h": rlk.gated_linear(x, w, s["act"])}
    if kind == "linear_train":
        y = rlk.det_linear_trainable(x, w, checkpoint="int8")
        grads = torch.autograd.grad(y, (x, w), s["grad"])
        return {"y": y.detach(), "grad_x": grads[0], "grad_weight": grads[1]}
    kept = None
    if s["hold"] == "again":
        h = rlk.gated_linear(x, w, s["act"])
    else:
        h, kept = rlk.gated_linear(x, w, s["act"], keep=s["hold"])
        if s["hold"] == "int8":
            x = rlk.unpack_int8(*rlk.pack_int8(x))
    grad_x, grad_weight = rlk.gated_linear_backward(s["grad"], x, w, s["act"], kept=kept)
    return {"h": h, "grad_x": grad_x, "grad_weight": grad_weight}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _exact_8_bits(x):
    """Rows of 64-bit numbers as their blocks hold them."""
    out = torch.zeros_like(x)
    for c in range(0, x.size(1), BLOCK):
        part = x[:, c:c + BLOCK]
        most = part.abs().amax(1, keepdim=True)
        power = (most / torch.frexp(most).mantissa).nan_to_num(0.0)           # above most, at most twice it
        step = (power / 128).clamp(min=2.0 ** -126)
        out[:, c:c + BLOCK] = torch.clamp(torch.round(part / step), -127, 127) * step
    return out


def _exact_act(g, act):
    if act == "silu":
        return torch.nn.functional.silu(g)
    return torch.nn.functional.gelu(g, approximate="tanh")


def exact(case, seed):
    s = prepare(case, seed)
    d, kind = torch.float64, case["kind"]
    if kind.startswith("embed"):
        ids, weight = s["ids"], s["weight"]
        one = torch.nn.functional.pad(weight, (0, 0, 0, 1))                   # a last row of zeros
        at = torch.where((ids < 0) | (ids >= case["vocab"]), case["vocab"], ids)
        out = {"out": one.index_select(0, at).to(d).mul_(case["scale"])}
        if kind == "embed_train":
            table = torch.zeros(one.shape, device="cuda", dtype=d)
            table.index_add_(0, at, s["grad"].to(d))
            out["grad_weight"] = table[:-1].mul_(case["scale"])
        return out
    if kind == "pack":
        return {"values": None, "exponents": None, "back": _exact_8_bits(s["x"].to(d))}
    x, w = s["x"].detach().to(d), s["weight"].detach().to(d)
    if kind == "linear_train":
        dy = s["grad"].to(d)
        return {"y": x.mm(w.T), "grad_x": dy.mm(w), "grad_weight": dy.T.mm(_exact_8_bits(x))}
    f = case["inner"]
    gate, up = x.mm(w[:f].T), x.mm(w[f:].T)
    out = {"h": _exact_act(gate, case["act"]) * up}
    if kind == "gated":
        return out
    if case["hold"] == "int8":
        gate, up, x = _exact_8_bits(gate), _exact_8_bits(up), _exact_8_bits(x)
    gate.requires_grad_()
    up.requires_grad_()
    dg, du = torch.autograd.grad(_exact_act(gate, case["act"]) * up, (gate, up), s["grad"].to(d))
    out["grad_x"] = dg.mm(w[:f]).addmm_(du, w[f:])
    out["grad_weight"] = torch.cat([dg.T.mm(x), du.T.mm(x)])
    return out
