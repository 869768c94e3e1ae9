"""min-p among near-equal logits: the weights' polynomial is rounded step by step, so the smaller of
two neighbouring logits can have the larger weight, and what min-p keeps need not be a prefix of the
sorted order."""
import numpy as np
import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
import sample_reference as ref
from helpers import cuda_or_skip

pytestmark = pytest.mark.gpu
LOG2E = np.float32(1.4426950408889634)


def inversions(n, lo=-0.72, hi=-0.1):
    """(higher logit, lower logit, weight of the lower) of neighbouring FP32 logits below a top of 0,
    the lower one heavier; n of them, the lightest first."""
    found = []
    for start in np.linspace(lo, hi, 4 * n).astype(np.float32):
        z = start.view(np.int32) - np.arange(4000, dtype=np.int32)     # upwards, towards 0
        z = z.view(np.float32)
        w = ref.weights(z, np.float32(0), LOG2E)
        at = np.nonzero((w[:-1] > w[1:]) & (w[:-1] % 128 == 0))[0]
        if len(at):
            found.append((z[at[0] + 1], z[at[0]], int(w[at[0]])))
        if len(found) == n:
            return found
    raise AssertionError("not enough inversions")


def rows(V, n, fill):
    """Rows of V logits: one top, n pairs at spread ids with the higher logit of each dropped by the
    row's min-p (that of one pair), which keeps the lower logit of that pair."""
    pairs = inversions(n)
    z = np.full((n, V), fill, np.float32)
    least = np.empty(n, np.float32)
    rng = np.random.default_rng(V)
    for r in range(n):
        ids = rng.permutation(V)[:2 * n + 1]
        z[r, ids[0]] = 0.0
        for i, (high, low, _) in enumerate(pairs):
            z[r, ids[1 + 2 * i]], z[r, ids[2 + 2 * i]] = high, low
        least[r] = np.float32(pairs[r][2] / 2 ** 31)
        assert int(np.rint(np.float64(least[r]) * 2 ** 24)) * 128 == pairs[r][2]
    return z, least


def check(dev, z, u, **how):
    n = len(z)
    put = {k: torch.from_numpy(v).to(dev) if isinstance(v, np.ndarray) else v for k, v in how.items()}
    token, logp = rlk.sample_logits(torch.from_numpy(z).to(dev), torch.from_numpy(u).to(dev), **put)
    assert rlk.device_error() == 0
    want, want_logp = ref.rows(z, u, **how)
    assert np.array_equal(token.cpu().numpy(), want)
    bound = ref.logp_bound(want_logp, z.shape[1], float(np.abs(z).max()) * 2, 1.0)
    assert (np.abs(logp.cpu().double().numpy() - want_logp) <= bound).all()
    assert len(want) == n


def test_reference_keeps_the_lower_of_a_pair():
    z, least = rows(64, 6, -50.0)
    dropped = 0
    for r in range(6):
        kept = ref.row(z[r], 0.5, 1.0, 20, 1.0, float(least[r]))[2]
        order = np.argsort(-z[r], kind="stable")
        places = np.sort(np.nonzero(np.isin(order, kept))[0])
        dropped += places[-1] != len(places) - 1       # not a prefix
    assert dropped == 6


@pytest.mark.parametrize("u", [0.0, 0.3, 0.9, 1.0 - 2.0 ** -31])
def test_one_pair(u):
    dev = cuda_or_skip()
    z = np.array([[0.0, -0.11424444615840912, -0.11424445360898972, -50.0]], np.float32)
    check(dev, z, np.array([u]), top_k=3, min_p=np.array([1915640960 / 2 ** 31], np.float32))


@pytest.mark.parametrize("how", [dict(top_k=20), dict(top_k=20, top_p=0.999), dict(top_p=0.999), dict()])
@pytest.mark.parametrize("V,copies,fill", [(64, 1, -50.0), (5003, 1, -50.0), (5003, 1, -12.0), (20011, 20, -50.0),
                                           (20011, 20, -12.0), (20011, 2, -50.0), (20011, 2, -12.0)])
def test_kept_sets_with_holes(V, copies, fill, how):
    """Short lists, rows by clusters and by the streaming kernels, and the passes that take every
    element by itself."""
    dev = cuda_or_skip()
    z, least = rows(V, 6, fill)
    z, least = np.tile(z, (copies, 1)), np.tile(least, copies)
    for u in (0.05, 0.5, 0.97, 1.0 - 2.0 ** -31):
        check(dev, z, np.full(len(z), u), min_p=least, **how)


def test_long_lists_with_holes():
    """More near-equal logits than the threads of a block: the list is ended by the block."""
    dev = cuda_or_skip()
    pairs = inversions(4)
    z = np.full((4, 9000), -50.0, np.float32)
    least = np.empty(4, np.float32)
    for r, (high, low, w) in enumerate(pairs):
        z[r, 5], z[r, 100:1500:2], z[r, 101:1500:2] = 0.0, high, low
        least[r] = np.float32(w / 2 ** 31)
    for how in (dict(top_k=1401), dict(top_k=1300, top_p=0.99), dict(top_p=0.999)):
        for u in (0.2, 0.8):
            check(dev, z, np.full(4, u), min_p=least, **how)
