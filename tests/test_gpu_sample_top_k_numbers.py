"""top_k as a Python number of any size, and what is not a whole number."""
import numpy as np
import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
from helpers import bits_equal, cuda_or_skip

pytestmark = pytest.mark.gpu


def test_numbers():
    dev = cuda_or_skip()
    g = torch.Generator(device=dev).manual_seed(0)
    z = torch.randn(30, 2000, device=dev, generator=g)
    u = torch.rand(30, device=dev, generator=g)
    every = rlk.sample_logits(z, u)
    for k in (2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 64 + 3, 2000, 0, -1, -2 ** 31 - 5, -2 ** 32 + 7):
        got = rlk.sample_logits(z, u, top_k=k)
        assert torch.equal(got[0], every[0]) and bits_equal(got[1], every[1]), k
    few = rlk.sample_logits(z, u, top_k=7)
    assert torch.equal(few[0], rlk.sample_logits(z, u, top_k=np.int64(7))[0])
    assert not torch.equal(few[0], every[0])
    with pytest.raises(TypeError):
        rlk.sample_logits(z, u, top_k=7.5)
