"""Measured cases of the sampling and distillation operators, with their plain forms.

``sample``  one token a row from [rows, vocab] logits: temperature, top-k, top-p
            and min-p, drawn with one given uniform number a row.
``distill`` the forward of a teacher's top logits against a linear student: loss
            and log-sum-exp a row, the [rows, vocab] logits never stored.
``train``   the same loss forward and backward: loss, log-sum-exp and the
            gradients of hidden, weight and (where there is one) bias.

Where ``own`` is false ``run`` computes a case with elementary torch operations;
where it is true it calls the framework.
"""
import math

import numpy as np
import torch

own = False

BF16_BYTES, FP32_BYTES, INT64_BYTES = 2, 4, 8


# ------------------------------------------------------------------ the cases
def _sample(name, rows, vocab, dtype, filters, uniform="fp32", pitch=0):
    return {"name": name, "kind": "sample", "rows": rows, "vocab": vocab, "dtype": dtype,
            "filters": filters, "uniform": uniform, "pitch": pitch}


def _distill(name, kind, rows, hidden, vocab, slots, bias=False, tau=1.0, padded=False, tail=False):
    return {"name": name, "kind": kind, "rows": rows, "hidden": hidden, "vocab": vocab,
            "slots": slots, "bias": bias, "tau": tau, "padded": padded, "tail": tail}


def listed():
    return [
        # one request being decoded, the usual settings: latency is all there is
        _sample("sample one row", 1, 151936, "fp32", "usual"),
        # a few rows of an odd vocabulary at an odd pitch, the whole distribution
        _sample("sample ragged", 7, 32003, "bf16", "none", "fp64", pitch=32011),
        # a decode batch whose requests each bring settings of their own
        _sample("sample mixed", 64, 151936, "fp32", "mixed", "fp64"),
        # rollout generation: many rows, one nucleus setting
        _sample("sample rollout", 512, 152064, "bf16", "nucleus"),
        # the widest decode batch, FP32 logits, each row its own settings
        _sample("sample wide", 1024, 151936, "fp32", "mixed", "fp64"),
        # the smallest student: launches and latency
        _distill("distill tiny", "distill", 64, 256, 1024, 8, bias=True),
        # scoring a handful of rows: the weight is streamed once
        _distill("distill 17 rows", "distill", 17, 4096, 151936, 64, tau=2.0, tail=True),
        # a scoring batch at the full vocabulary, ragged teacher lists
        _distill("distill batch", "distill", 4096, 4096, 151936, 64, padded=True),
        # training step of the smallest student
        _distill("train tiny", "train", 64, 256, 1024, 8, bias=True, tau=2.0),
        # a short odd batch with a bias and ragged lists
        _distill("train ragged", "train", 255, 2048, 32003, 33, bias=True, padded=True),
        # a micro-batch of an ordinary student
        _distill("train middle", "train", 1024, 2048, 32003, 20, tau=1.5, tail=True),
        # a micro-batch at the full vocabulary
        _distill("train batch", "train", 2048, 4096, 151936, 64, padded=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["sample", "sample", "distill", "train"])
    vocab = _log_int(rng, 1000, 152064)
    if kind == "sample":
        rows = min(_log_int(rng, 1, 1024), 1024 * 151936 // vocab)
        pitch = rng.choice([0, 0, vocab + rng.randrange(1, 9)])
        return {k: v for k, v in _sample("", rows, vocab, rng.choice(["fp32", "bf16"]),
                                         rng.choice(["none", "usual", "nucleus", "mixed"]),
                                         rng.choice(["fp32", "fp64"]), pitch).items() if k != "name"}
    hidden = rng.choice([256, 512, 1000, 1024, 1537, 2048, 4096])
    most = 4096 * 4096 * 151936 if kind == "distill" else 2048 * 4096 * 151936
    rows = min(_log_int(rng, 1, 4096), most // (hidden * vocab))
    c = _distill("", kind, rows, hidden, vocab, _log_int(rng, 1, 128), rng.random() < 0.5,
                 rng.choice([1.0, 1.0, 1.5, 2.0]), rng.random() < 0.5, rng.random() < 0.5)
    return {k: v for k, v in c.items() if k != "name"}


def work(case):
    n, v = case["rows"], case["vocab"]
    if case["kind"] == "sample":
        size = FP32_BYTES if case["dtype"] == "fp32" else BF16_BYTES
        draws = FP32_BYTES if case["uniform"] == "fp32" else INT64_BYTES
        each = draws + INT64_BYTES + FP32_BYTES + (16 if case["filters"] == "mixed" else 0)
        return {"bytes": n * v * size + n * each, "flops": 4 * n * v}
    h, k = case["hidden"], case["slots"]
    read = BF16_BYTES * (n + v) * h + n * k * (INT64_BYTES + FP32_BYTES)
    read += FP32_BYTES * (v * case["bias"] + n * case["tail"])
    wrote = 2 * FP32_BYTES * n
    flops = 2 * n * h * v
    if case["kind"] == "train":       # the upstream gradient, then both products and the bias sum
        read += FP32_BYTES * n
        wrote += BF16_BYTES * (n + v) * h + FP32_BYTES * v * case["bias"]
        flops *= 3
    return {"bytes": read + wrote, "flops": flops}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _pick(values, n, g, dtype):
    return torch.tensor(values, device="cuda", dtype=dtype)[
        torch.randint(len(values), (n,), device="cuda", generator=g)]


def _prepare_sample(case, seed):
    g = _generator(seed)
    n, v = case["rows"], case["vocab"]
    pitch = case["pitch"] or v
    dtype = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    # a bulk of unlikely ids under a short head whose lead differs from row to row
    # (confident rows and open ones), and the last ids of the vocabulary banned
    z = torch.randn(n, pitch, device="cuda", generator=g).mul_(1.5)
    heads = min(96, v // 4)
    at = torch.randint(v, (n, heads), device="cuda", generator=g)
    top = torch.rand(n, 1, device="cuda", generator=g) * 10 + 12
    fall = torch.rand(n, 1, device="cuda", generator=g) * 1.5 + 0.8
    rank = torch.arange(1, heads + 1, device="cuda", dtype=torch.float32).log()
    z.scatter_reduce_(1, at, top - fall * rank + torch.rand(n, heads, device="cuda", generator=g),
                      "amax")
    z[:, v - v // 64:] = -math.inf
    s = {"kind": "sample", "logits": z.to(dtype)[:, :v],
         "uniform": torch.rand(n, device="cuda", generator=g,
                               dtype=torch.float32 if case["uniform"] == "fp32" else torch.float64)}
    if case["filters"] == "mixed":
        s["how"] = {"temperature": _pick([0.0, 0.6, 0.8, 1.0, 1.2], n, g, torch.float32),
                    "top_k": _pick([0, 1, 20, 50, 200], n, g, torch.int32),
                    "top_p": _pick([0.5, 0.9, 0.95, 1.0], n, g, torch.float32),
                    "min_p": _pick([0.0, 0.0, 0.02, 0.1], n, g, torch.float32)}
    else:
        s["how"] = {"none": {}, "usual": {"temperature": 0.8, "top_k": 50, "top_p": 0.95},
                    "nucleus": {"temperature": 1.0, "top_p": 0.95}}[case["filters"]]
    return s


def _prepare_distill(case, seed):
    g = _generator(seed)
    n, h, v, k = (case[x] for x in ("rows", "hidden", "vocab", "slots"))
    hidden = torch.randn(n, h, device="cuda", generator=g).bfloat16()
    weight = torch.randn(v, h, device="cuda", generator=g).mul_(2.5 / math.sqrt(h)).bfloat16()
    bias = torch.randn(v, device="cuda", generator=g).mul_(0.1) if case["bias"] else None
    # the teacher: a related model's logits, of which the largest are kept
    ids, logits, lse = [], [], []
    for r in range(0, n, 512):
        z = (hidden[r:r + 512] @ weight.t()).float()
        z += torch.randn(z.shape, device="cuda", generator=g).mul_(2.0)
        best = z.topk(k, dim=1)
        ids.append(best.indices)
        logits.append(best.values)
        lse.append(torch.logsumexp(z / case["tau"], 1))
    ids, logits, lse = torch.cat(ids), torch.cat(logits), torch.cat(lse)
    if case["padded"]:                # lists of unequal length, some rows without any
        length = torch.randint(k + 1, (n, 1), device="cuda", generator=g)
        length = torch.where(torch.rand(n, 1, device="cuda", generator=g) < 0.7, k, length)
        slot = torch.arange(k, device="cuda")
        ids = torch.where(slot < length, ids, -1)
        logits = torch.where(slot < length, logits, -math.inf)
    s = {"kind": case["kind"], "hidden": hidden, "weight": weight, "bias": bias, "ids": ids,
         "logits": logits, "tau": case["tau"], "teacher_lse": lse if case["tail"] else None}
    if case["kind"] == "train":
        s["grad"] = torch.rand(n, device="cuda", generator=g).add_(0.5).div_(n)
        for t in (hidden, weight, bias):
            if t is not None:
                t.requires_grad_()
    return s


def prepare(case, seed):
    return (_prepare_sample if case["kind"] == "sample" else _prepare_distill)(case, seed)


# ------------------------------------------------------------------ sampling, the plain form
# A weight is 2^x rounded to a multiple of 2^-31, where x = (z - max z) log2(e) / T:
# 2^x = 2^n 2^f with n the nearest whole number, and 2^f by this polynomial on
# [-1/2, 1/2] (least-squares fit of the relative error, which it keeps under 2e-7),
# each product and each sum rounded to 32 bits.  Every sum after that is of whole
# numbers, so the token is one definite number whatever the order of the sums.
EXP2 = (0.0013264727313071489, 0.009671512991189957, 0.05550733581185341, 0.24022242426872253,
        0.6931470036506653, 1.0)
LOG2E = 1.4426950408889634
GREEDY_BELOW = 1e-6
ONE = 1 << 31
FRACTION = 1 << 24


def _rows(value, n, dtype):
    value = torch.as_tensor(value, dtype=dtype, device="cuda")
    return value.expand(n).reshape(n, 1)


def _whole(value):                     # a share in [0, 1] as a multiple of 2^-24
    return (value.clamp(0, 1) * FRACTION).round().to(torch.int64)


def _weights(z, top, scale):
    x = ((z - top) * scale).clamp_(min=-126.0)
    n = torch.round(x)
    f = x.sub_(n)
    y = torch.full_like(f, EXP2[0])
    for c in EXP2[1:]:
        y = y.mul_(f).add_(c)
    power = ((n.to(torch.int32) + (127 + 31)) << 23).view(torch.float32)
    return y.mul_(power).round_().to(torch.int64)


def _plain_sample(s):
    z = s["logits"].float() + 0.0
    n, v = z.shape
    how = s["how"]
    tau = _rows(how.get("temperature", 1.0), n, torch.float32)
    top_k = _rows(how.get("top_k", 0), n, torch.int64)
    greedy = tau < GREEDY_BELOW
    tau = torch.where(greedy, 1.0, tau)
    top_k = torch.where(greedy, 1, torch.where(top_k > 0, top_k, v))
    top_p = _whole(_rows(how.get("top_p", 1.0), n, torch.float32))
    least = _whole(_rows(how.get("min_p", 0.0), n, torch.float32)) << 7
    top = z.amax(1, keepdim=True)
    w = _weights(z, top, torch.tensor(LOG2E, device="cuda") / tau)
    # from the largest logit down, equal ones by id
    order = torch.sort(z, dim=1, descending=True, stable=True).indices
    ranked = w.gather(1, order) * (torch.arange(v, device="cuda") < top_k)
    before = ranked.cumsum(1)
    total = before[:, -1:]
    most = ((top_p * (total >> 31)) << 7) + ((top_p * (total & (ONE - 1))) >> 24)
    before -= ranked
    ranked *= (before < most.clamp(min=1)) & (ranked >= least)
    w.scatter_(1, order, ranked)
    upto = w.cumsum(1)                 # by id
    total = upto[:, -1:]
    u = (s["uniform"].reshape(n, 1).double() * ONE).floor().to(torch.int64)
    at = u * (total >> 31) + ((u * (total & (ONE - 1))) >> 31)
    token = (upto <= at).sum(1, keepdim=True)
    logp = (z.gather(1, token) - top) / tau - torch.log(total.float() / ONE)
    return {"token": token.reshape(n), "logp": logp.reshape(n)}


# ------------------------------------------------------------------ distillation, the plain form
def _plain_teacher(s):
    ids, a = s["ids"], s["logits"].float() / s["tau"]
    used = (ids >= 0) & (ids < s["weight"].size(0)) & (a > -math.inf)
    a = torch.where(used, a, -math.inf)
    if s["teacher_lse"] is None:
        top = a.amax(1, keepdim=True).clamp(min=-1e30)
        norm = top + (a - top).exp().sum(1, keepdim=True).log()
    else:
        norm = s["teacher_lse"].reshape(-1, 1)
    logq = torch.where(used, a - norm, 0.0)
    return torch.where(used, ids, 0), logq, torch.where(used, logq.exp(), 0.0)


def _plain_distill(s):
    tau = s["tau"]
    hidden, weight = s["hidden"].detach().float(), s["weight"].detach().float()
    z = hidden @ weight.t()
    if s["bias"] is not None:
        z += s["bias"].detach()
    z /= tau
    top = z.amax(1, keepdim=True)
    p = (z - top).exp_()
    total = p.sum(1, keepdim=True)
    lse = top + total.log()
    ids, logq, q = _plain_teacher(s)
    loss = tau * tau * (q * (logq - z.gather(1, ids) + lse)).sum(1)
    out = {"loss": loss, "lse": lse.reshape(-1)}
    if s["kind"] == "distill":
        return out
    grad = p.mul_(q.sum(1, keepdim=True) / total)
    grad.scatter_add_(1, ids, -q)
    grad *= tau * s["grad"].reshape(-1, 1)
    out["grad_hidden"] = (grad @ weight).bfloat16()
    out["grad_weight"] = (grad.t() @ hidden).bfloat16()
    if s["bias"] is not None:
        out["grad_bias"] = grad.sum(0)
    return out


# ------------------------------------------------------------------ one pass
def run(state):
    if not own:
        with torch.no_grad():
            return (_plain_sample if state["kind"] == "sample" else _plain_distill)(state)
    import deterministic_invariant_gemm_linear_gb300 as rlk
    if state["kind"] == "sample":
        token, logp = rlk.sample_logits(state["logits"], state["uniform"], **state["how"])
        return {"token": token, "logp": logp}
    hidden, weight, bias = state["hidden"], state["weight"], state["bias"]
    if state["kind"] == "distill":
        loss, lse = rlk.linear_distill(hidden, weight, state["ids"], state["logits"], bias,
                                       temperature=state["tau"], teacher_lse=state["teacher_lse"])
        return {"loss": loss, "lse": lse}
    loss, lse = rlk.linear_distill_trainable(hidden, weight, state["ids"], state["logits"], bias,
                                             temperature=state["tau"],
                                             teacher_lse=state["teacher_lse"])
    inputs = [t for t in (hidden, weight, bias) if t is not None]
    grads = torch.autograd.grad(loss, inputs, state["grad"])
    out = {"loss": loss.detach(), "lse": lse, "grad_hidden": grads[0], "grad_weight": grads[1]}
    if bias is not None:
        out["grad_bias"] = grads[2]
    return out


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _exact_row(z, u, tau, top_k, top_p, min_p):
    """The token by whole-number arithmetic on the defined weights, and its exact log-probability."""
    one = np.float32
    if tau < one(GREEDY_BELOW):
        tau, top_k = one(1), 1
    top = z.max()
    with np.errstate(over="ignore"):
        x = np.maximum((z - top) * (one(LOG2E) / tau), one(-126))
    n = np.rint(x)
    f = x - n
    y = np.full_like(f, one(EXP2[0]))
    for c in EXP2[1:]:
        y = y * f + one(c)
    w = np.rint(np.ldexp(y.astype(np.float64), n.astype(np.int64) + 31)).astype(np.int64)
    kept = np.argsort(-z, kind="stable")
    if top_k > 0:
        kept = kept[:top_k]
    upto = np.cumsum(w[kept])
    most = max(1, int(round(float(min(max(top_p, 0), 1)) * FRACTION)) * int(upto[-1]) // FRACTION)
    kept = kept[upto - w[kept] < most]
    kept = np.sort(kept[w[kept] >= int(round(float(min(max(min_p, 0), 1)) * FRACTION)) << 7])
    upto = np.cumsum(w[kept])
    token = kept[np.searchsorted(upto, int(u * ONE) * int(upto[-1]) // ONE, side="right")]
    p = np.exp((z[kept].astype(np.float64) - float(top)) / float(tau))
    return token, (float(z[token]) - float(top)) / float(tau) - math.log(p.sum())


def _exact_sample(case, seed):
    if case["rows"] * case["vocab"] > 40_000_000:
        return None
    s = _prepare_sample(case, seed)
    n = case["rows"]
    z = s["logits"].float().cpu().numpy()
    u = s["uniform"].double().cpu().numpy()
    how = [np.broadcast_to(s["how"][k].cpu().numpy() if torch.is_tensor(s["how"].get(k))
                           else np.asarray(s["how"].get(k, d), t), (n,))
           for k, d, t in (("temperature", 1.0, np.float32), ("top_k", 0, np.int64),
                           ("top_p", 1.0, np.float32), ("min_p", 0.0, np.float32))]
    got = [_exact_row(z[r], u[r], *[x[r] for x in how]) for r in range(n)]
    return {"token": np.array([t for t, _ in got], np.int64), "logp": np.array([p for _, p in got])}


def _exact_distill(case, seed):
    s = _prepare_distill(case, seed)
    d = torch.float64
    tau, (n, k) = case["tau"], s["ids"].shape
    x = s["hidden"].detach().to(d)
    w = s["weight"].detach().to(d)
    z = torch.mm(x, w.T)
    if s["bias"] is not None:
        z = z + s["bias"].detach().to(d)
    logp = torch.log_softmax(z / tau, 1)
    lse = z[:, 0] / tau - logp[:, 0]
    # the teacher as a sparse row over the vocabulary; rows of no slots keep zeros
    ids, a = s["ids"], s["logits"].to(d) / tau
    none = (ids < 0) | (ids >= case["vocab"])
    a = a.masked_fill(none, -math.inf)
    norm = torch.logsumexp(a, 1) if s["teacher_lse"] is None else s["teacher_lse"].to(d)
    norm = torch.where(none.all(1), 0.0, norm)
    q = torch.exp(a - norm[:, None])
    cross = torch.where(q > 0, q * (a - norm[:, None] - logp.gather(1, ids.clamp(min=0))), 0.0)
    out = {"loss": tau ** 2 * cross.nan_to_num(0.0).sum(1), "lse": lse}
    if case["kind"] == "distill":
        return out
    dz = logp.exp_().mul_(q.sum(1)[:, None])
    dz.scatter_add_(1, ids.clamp(min=0), -q)
    dz.mul_(s["grad"].to(d)[:, None] * tau)
    out["grad_hidden"] = torch.mm(dz, w)
    out["grad_weight"] = torch.mm(dz.T, x)
    if s["bias"] is not None:
        out["grad_bias"] = dz.sum(0)
    return out


def exact(case, seed):
    with torch.no_grad():
        return (_exact_sample if case["kind"] == "sample" else _exact_distill)(case, seed)
