"""The 64-bit distillation reference against torch's own routines and finite differences."""
import math

import pytest
import torch

import distill_reference as ref


def case(N, H, V, K, seed=0, bias=True):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(N, H, generator=g)
    w = torch.randn(V, H, generator=g) * (2 / math.sqrt(H))
    b = torch.randn(V, generator=g) * 0.1 if bias else None
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(N)])
    return h, w, ids, torch.randn(N, K, generator=g) * 2, b


@pytest.mark.parametrize("T", [1.0, 2.0])
def test_loss_is_the_kl_divergence(T):
    h, w, ids, t, b = case(5, 7, 11, 11)
    z = h.double() @ w.double().T + b.double()
    full = torch.empty(5, 11, dtype=torch.float64).scatter_(1, ids, t.double())
    want = T ** 2 * torch.nn.functional.kl_div(torch.log_softmax(z / T, 1),
                                               torch.softmax(full / T, 1), reduction="none").sum(1)
    loss, lse = ref.distill(h, w, ids, t, b, T)
    assert torch.allclose(loss, want, rtol=1e-12, atol=1e-12)
    assert torch.allclose(lse, torch.logsumexp(z / T, 1), rtol=1e-13)


@pytest.mark.parametrize("T", [1.0, 0.5])
@pytest.mark.parametrize("tail", [False, True])
def test_gradient_against_differences(T, tail):
    h, w, ids, t, b = (x.double() if x.is_floating_point() else x for x in case(4, 6, 19, 5))
    ids[1, 2:] = -1                       # a short list
    ids[2, :] = 19                        # none at all
    ids[3, 1] = ids[3, 0]                 # an id named twice
    tl = torch.logsumexp(t / T, 1) + 0.3 if tail else None
    g = torch.tensor([1.0, -2.0, 3.0, 0.5], dtype=torch.float64)
    G = ref.grad_logits(h, w, ids, t, g, b, T, tl)
    assert torch.equal(G[2], torch.zeros(19, dtype=torch.float64))
    for x, dx in ((h, G @ w), (w, G.T @ h), (b, G.sum(0))):
        d = torch.randn(x.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(3))
        eps = 1e-6
        keep = x.clone()
        x.copy_(keep + eps * d)
        up = (g * ref.distill(h, w, ids, t, b, T, tl)[0]).sum()
        x.copy_(keep - eps * d)
        down = (g * ref.distill(h, w, ids, t, b, T, tl)[0]).sum()
        x.copy_(keep)
        assert (up - down) / (2 * eps) == pytest.approx((dx * d).sum().item(), rel=1e-6, abs=1e-8)
