"""Kept logits handed to the backward in other layouts than the forward's own give its bits."""
import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
from helpers import bits_equal, cuda_or_skip

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1, 5])
@pytest.mark.parametrize("V", [1001, 1008])
def test_layouts_of_kept_logits(N, V):
    dev = cuda_or_skip()
    g = torch.Generator(device=dev).manual_seed(N)
    h = torch.randn(N, 40, device=dev, generator=g).bfloat16()
    w = torch.randn(V, 40, device=dev, generator=g).bfloat16()
    ids = torch.randint(V, (N, 6), device=dev, generator=g)
    t = torch.randn(N, 6, device=dev, generator=g)
    up = torch.randn(N, device=dev, generator=g)
    loss, lse, z = rlk.linear_distill(h, w, ids, t, return_logits=True)
    want = rlk.linear_distill_backward(h, w, ids, t, lse, up)
    wide = torch.zeros(N, V + 21, device=dev)
    wide[:, 3:3 + V] = z
    for kept in (z, z.clone(), z.contiguous().clone(), wide[:, 3:3 + V], z.t().contiguous().t()):
        got = rlk.linear_distill_backward(h, w, ids, t, lse, up, logits=kept)
        assert bits_equal(got[0], want[0]) and bits_equal(got[1], want[1])
    with pytest.raises(ValueError):
        rlk.linear_distill_backward(h, w, ids, t, lse, up, logits=z.bfloat16())
    assert rlk.device_error() == 0
