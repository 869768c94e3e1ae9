"""One token a row by the sampling operator's definition, with numpy's FP32 operations and
Python's whole numbers: the sort, the running sums and the products are all exact."""
import math

import numpy as np

F = np.float32
COEFFS = (0.0013264727313071489, 0.009671512991189957, 0.05550733581185341, 0.24022242426872253,
          0.6931470036506653, 1.0)


def weights(z, top, c):
    """Whole-number weights 2^31 2^x of FP32 logits."""
    with np.errstate(over="ignore"):
        x = np.maximum((z - top).astype(F) * F(c), F(-126))
    n = np.rint(x)
    f = (x - n).astype(F)
    y = np.full_like(f, F(COEFFS[0]))
    for a in COEFFS[1:]:
        y = (y * f).astype(F) + F(a)
    return np.rint(np.ldexp(y.astype(np.float64), n.astype(np.int64) + 31)).astype(np.int64)


def part(p):
    return int(np.rint(float(F(min(max(p, 0.0), 1.0))) * 2 ** 24))


def row(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logp in 64 bits, kept ids); (-1, nan, none) where there is no distribution."""
    z = np.asarray(z, F)
    tau = F(temperature)
    if any(x != x for x in (tau, top_p, min_p, u)) or not 0 <= tau < np.inf or \
            np.isnan(z).any() or (z == np.inf).any() or (z == -np.inf).all():
        return -1, math.nan, np.zeros(0, np.int64)
    if tau < F(1e-6):
        tau, top_k = F(1), 1
    top = z.max()
    w = weights(z, top, F(1.4426950408889634) / tau)
    order = np.argsort(-z.astype(np.float64), kind="stable")
    if 0 < top_k < len(z):
        order = order[:top_k]
    total = sum(int(x) for x in w[order])
    most = max(1, part(top_p) * total // 2 ** 24)
    before = np.cumsum(w[order]) - w[order]
    kept = order[before < most]
    kept = np.sort(kept[w[kept] >= part(min_p) * 128])
    upto = np.cumsum(w[kept])
    u31 = min(max(int(math.floor(u * 2.0 ** 31)), 0), 2 ** 31 - 1)
    at = u31 * int(upto[-1]) // 2 ** 31
    token = int(kept[np.searchsorted(upto, at, side="right")])
    x = (z[kept].astype(np.float64) - float(top)) / float(tau)
    return token, (float(z[token]) - float(top)) / float(tau) - math.log(np.exp(x).sum()), kept


def rows(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    n = len(z)
    how = [np.broadcast_to(np.asarray(x), (n,)) for x in (temperature, top_k, top_p, min_p)]
    out = [row(z[i], float(u[i]), float(how[0][i]), int(how[1][i]), float(how[2][i]),
               float(how[3][i])) for i in range(n)]
    return np.array([o[0] for o in out]), np.array([o[1] for o in out])


# logp against 64 bits: the weights' relative error (2e-7 and half a step of 2^-31, V of
# them), the FP32 rounding of (z - m), of the quotient and of the logarithm.
def logp_bound(logp, V, spread, temperature):
    return 2e-6 + V * 2.0 ** -32 + 2.0 ** -22 * (np.abs(logp) + spread / max(temperature, 1e-6))
