"""The sampling reference against distributions computed another way, and its edges."""
import math

import numpy as np
import pytest

import sample_reference as ref


def kept_by_sorting(z, T, k, p, m):
    """The kept set from 64-bit probabilities."""
    q = np.exp((z.astype(np.float64) - z.max()) / T)
    order = np.argsort(-z, kind="stable")
    if 0 < k < len(z):
        order = order[:k]
    before = np.cumsum(q[order]) - q[order]
    order = order[before < max(p * q[order].sum(), 1e-300)]
    return np.sort(order[q[order] >= m])


@pytest.mark.parametrize("T,k,p,m", [(1.0, 0, 1.0, 0.0), (0.7, 40, 1.0, 0.0), (1.3, 0, 0.9, 0.0),
                                     (1.0, 0, 1.0, 0.07), (0.9, 33, 0.8, 0.02), (1.0, 1, 0.5, 0.3)])
def test_frequencies_follow_the_distribution(T, k, p, m):
    rng = np.random.default_rng(1)
    z = (rng.standard_normal(300) * 2).astype(np.float32)
    tau = float(np.float32(T))              # the operator's temperature is FP32
    want = kept_by_sorting(z, tau, k, p, m)
    assert np.array_equal(ref.row(z, 0.3, T, k, p, m)[2], want)
    q = np.exp(z[want].astype(np.float64) / tau)
    edges = np.concatenate([[0], np.cumsum(q) / q.sum()])
    for u in rng.random(200):
        token, logp, _ = ref.row(z, u, T, k, p, m)
        i = np.searchsorted(want, token)
        assert edges[i] - 1e-6 <= u <= edges[i + 1] + 1e-6
        assert logp == pytest.approx(math.log(edges[i + 1] - edges[i]), abs=1e-9)


def test_edges():
    z = np.array([1, 3, 3, -math.inf, 2], np.float32)
    assert ref.row(z, 0.9, 0.0)[:2] == (1, 0.0)             # greedy: the lowest id of equal ones
    assert ref.row(z, 0.0, 1.0, 0, 0.0)[:2] == (1, 0.0)     # top-p 0 keeps one
    assert list(ref.row(z, 0.5, 1.0, 2)[2]) == [1, 2]
    assert list(ref.row(z, 0.5, 1.0, 0, 1.0, 1.0)[2]) == [1, 2]
    assert ref.row(z, 0.999999, 1.0)[0] == 4                # a banned id is never the last
    assert ref.row(np.full(3, -math.inf, np.float32), 0.5)[0] == -1
    assert ref.row(np.array([1, math.nan], np.float32), 0.5)[0] == -1
    assert ref.row(np.array([1, math.inf], np.float32), 0.5)[0] == -1
    assert ref.row(z, 0.5, math.nan)[0] == -1 and ref.row(z, 0.5, -1.0)[0] == -1
    assert ref.row(z[:1], 0.7)[:2] == (0, 0.0)


def test_weights_are_two_to_the_x():
    z = np.linspace(-40, 0, 100001).astype(np.float32)
    w = ref.weights(z, np.float32(0), np.float32(1.4426950408889634))
    exact = np.exp(z.astype(np.float64)) * 2 ** 31
    # 2e-7 of the polynomial and its roundings, 2^-24 |x| of the FP32 product, half a step
    assert (np.abs(w - exact) <= exact * (2e-7 + 60 * 2.0 ** -24) + 0.5).all()
    assert w[-1] == 2 ** 31 and (np.diff(w) >= -1).all()
