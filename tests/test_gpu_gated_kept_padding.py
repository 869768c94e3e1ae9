"""Kept projections past column F are zeros, whatever the rows hold."""
import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
from helpers import bits_equal, cuda_or_skip

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [20, 100, 140])        # both rings of the one-CTA loop, the 2-SM loop
@pytest.mark.parametrize("F", [1, 33, 100, 129])
def test_padding_of_rows_with_numbers_that_are_not_finite(M, F):
    dev = cuda_or_skip()
    g = torch.Generator(device=dev).manual_seed(F)
    x = torch.randn(M, 64, device=dev, generator=g).bfloat16()
    w = torch.randn(2 * F, 64, device=dev, generator=g).bfloat16()
    x[7, 3], x[11, 0], x[13, 5] = float("nan"), float("inf"), float("-inf")
    _, kept = rlk.gated_linear(x, w, keep="fp32")
    _, (q, _) = rlk.gated_linear(x, w, keep="int8")
    assert not kept[:, :, F:].any() and not q[:, :, F:].any()      # a NaN counts as true
    z = rlk.det_linear(x, w, torch.float32)
    assert bits_equal(kept[:, 0, :F] + 0.0, z[:, :F] + 0.0) and bits_equal(kept[:, 1, :F] + 0.0, z[:, F:] + 0.0)
    assert rlk.device_error() == 0
