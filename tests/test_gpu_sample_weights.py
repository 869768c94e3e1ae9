"""The weights themselves, to the last unit: a row of two logits draws the first exactly while the
uniform number is below a threshold that its weight gives, and the token just below and at that
threshold tells the weight to a unit or two."""
import numpy as np
import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
import sample_reference as ref
from helpers import cuda_or_skip

pytestmark = pytest.mark.gpu
LOG2E = np.float32(1.4426950408889634)
ONE = 1 << 31


def thresholds(w):
    """The least whole u with floor(u (2^31 + w) / 2^31) >= w."""
    return np.array([-(-int(x) * ONE // (ONE + int(x))) for x in w], np.int64)


def logits(n, seed):
    rng = np.random.default_rng(seed)
    z = -np.concatenate([rng.random(n // 2) * 1.5, rng.random(n - n // 2) * 22]).astype(np.float32)
    z[:3] = 0.0, -0.11424444615840912, -0.11424445360898972
    return z


@pytest.mark.parametrize("how", [dict(), dict(top_k=2), dict(top_p=1 - 2.0 ** -24), dict(min_p=2.0 ** -24)])
@pytest.mark.parametrize("temperature", [1.0, 0.7, 3.0])
@pytest.mark.parametrize("N,V", [(4096, 2), (300, 3001), (272, 16384)])
def test_weights(N, V, temperature, how):
    dev = cuda_or_skip()
    z = logits(N, V)
    c = LOG2E / np.float32(temperature)
    w = ref.weights(z, np.float32(0), c)
    rows = torch.full((N, V), -float("inf"))
    rows[:, 0], rows[:, 1] = torch.from_numpy(z), 0.0
    rows = rows.to(dev)
    u = thresholds(w)
    # what cuts drop does not draw: keep the rows whose lighter logit stays
    some = slice(None) if "top_p" not in how and "min_p" not in how else np.nonzero(w >= 2 ** 12)[0]
    for step, token in ((-1, 0), (0, 1)):
        x = torch.from_numpy(np.clip(u + step, 0, ONE - 1) / ONE).to(dev)
        got, _ = rlk.sample_logits(rows, x, temperature=temperature, **how)
        got = got.cpu().numpy()
        ok = (u + step >= 0) & (u + step < ONE)
        wrong = np.nonzero((got != token) & ok)[0]
        wrong = np.intersect1d(wrong, np.arange(N)[some])
        assert len(wrong) == 0, (len(wrong), z[wrong[:3]], w[wrong[:3]])
    assert rlk.device_error() == 0
