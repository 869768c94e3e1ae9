"""Teacher lists of many slots in a small vocabulary: hundreds of terms meet in one vocabulary split,
and the loss keeps the error bound of short lists."""
import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
import distill_reference as ref
from helpers import cuda_or_skip
from test_gpu_distill_precision import bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [0.5, 1.0, 1.5, 10.0])
@pytest.mark.parametrize("N,V,K", [(100, 5, 800), (100, 264, 900), (300, 31, 1024), (300, 1, 600)])
@pytest.mark.parametrize("tail", [False, True])
def test_long_lists(N, V, K, T, tail):
    dev = cuda_or_skip()
    g = torch.Generator().manual_seed(K)
    h = torch.randint(-6, 7, (N, 8), generator=g).bfloat16()
    w = (torch.randint(-4, 5, (V, 8), generator=g).float() / 4).bfloat16()      # exact logits, up to 40
    ids = torch.randint(V, (N, K), generator=g)
    t = (h.float() @ w.float().T).gather(1, ids) + torch.randn(N, K, generator=g) * 0.1
    tl = (torch.logsumexp(t.double() / T, 1) + 0.1).float() if tail else None
    want, _ = ref.distill(h, w, ids, t, None, T, tl)
    d = [x.to(dev) for x in (h, w, ids, t)]
    loss, _ = rlk.linear_distill(*d, temperature=T, teacher_lse=None if tl is None else tl.to(dev))
    error = (loss.cpu().double() - want).abs()
    limit = bound(h, w, ids, t, T, tl)
    assert (error <= limit).all(), (error / limit).max()
