"""top-k rows that hold NaN or +inf, or bring broken settings, in any CTA of a row's cluster: no token
for them, the definition's token for the rows beside them."""
import math

import numpy as np
import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
import sample_reference as ref
from helpers import cuda_or_skip

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,V", [(3, 700), (6, 40000), (6, 151936), (160, 20011)])
@pytest.mark.parametrize("k", [1, 40, 700])
def test_broken_rows(N, V, k):
    dev = cuda_or_skip()
    g = torch.Generator().manual_seed(N)
    z = torch.randn(N, V, generator=g) * 2
    tau = torch.full((N,), 0.8)
    bad = []
    for r in range(0, N, 2):
        kind = (r // 2) % 5
        at = (0, V - 1, V // 2, V // 3, 5)[kind]
        if kind == 2:
            tau[r] = math.nan
        elif kind == 4:
            z[r] = -math.inf
            z[r, at] = math.nan
        else:
            z[r, at] = (math.nan, math.inf, 0.0, math.nan)[kind]
        bad.append(r)
    u = torch.rand(N, generator=g, dtype=torch.float64)
    token, logp = rlk.sample_logits(z.to(dev), u.to(dev), temperature=tau.to(dev), top_k=k)
    assert rlk.device_error() == 0
    want, _ = ref.rows(z.numpy(), u.numpy(), tau.numpy(), k)
    assert np.array_equal(token.cpu().numpy(), want)
    assert (token.cpu()[bad] == -1).all() and torch.isnan(logp.cpu()[bad]).all()
    assert torch.isfinite(logp).sum() == N - len(bad)
