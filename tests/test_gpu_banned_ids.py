"""A bias of -inf bans ids, wherever they lie: the fused log-sum-exp, log-probability, distillation
loss and gradients against 64 bits; a row of NaN logits is not hidden."""
import math

import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
import distill_reference as ref
from helpers import bits_equal, cuda_or_skip

pytestmark = pytest.mark.gpu


def case(N, V, banned, seed=0, H=64):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(N, H, generator=g).bfloat16()
    w = (torch.randn(V, H, generator=g) * (2 / math.sqrt(H))).bfloat16()
    b = torch.randn(V, generator=g) * 0.1
    b[banned(V)] = -math.inf
    return h, w, b


BANNED = {
    "the first 32": lambda V: slice(0, 32),
    "the first 300": lambda V: slice(0, 300),
    "the last": lambda V: slice(V - 40, V),
    "all but one": lambda V: [v for v in range(V) if v != V // 2 + 3],
    "every second": lambda V: slice(0, V, 2),
    "whole tiles": lambda V: slice(256, 768),
}


def logit_bounds(h, w, b, T):
    """lse's bound as in distill_reference.bounds, over the allowed ids."""
    ok = torch.isfinite(b)
    z = h.double() @ w[ok].double().T + b[ok].double()
    dz = ref.logit_error(h, w[ok], b[ok]) / T
    lse = torch.logsumexp(z / T, 1)
    return z, lse, dz + 2.0 ** -20 * ((z / T).abs().amax(1) + lse.abs() + 1)


@pytest.mark.parametrize("banned", BANNED)
@pytest.mark.parametrize("N", [5, 100, 200])
def test_linear_logp(N, banned):
    dev = cuda_or_skip()
    V = 1500
    h, w, b = case(N, V, BANNED[banned])
    target = torch.randint(V, (N,), generator=torch.Generator().manual_seed(1))
    z, want, bound = logit_bounds(h, w, b, 1.0)
    hd, wd, bd, td = (x.to(dev) for x in (h, w, b, target))
    logp, lse = rlk.linear_logp(hd, wd, td, bd)
    assert ((lse.cpu().double() - want).abs() <= bound).all()
    allowed = torch.isfinite(b)[target]
    zt = (h.double() * w[target].double()).sum(1) + b[target].double()
    assert (logp.cpu()[~allowed] == -math.inf).all()
    assert ((logp.cpu().double() - (zt - want))[allowed].abs() <= 2 * bound[allowed]).all()
    gh, gw, gb, G = rlk.linear_logp_backward(hd, wd, td, lse, torch.ones(N, device=dev), bd,
                                             return_grad_logits=True)
    want_G = -torch.softmax(h.double() @ w.double().T + b.double(), 1)
    want_G[torch.arange(N), target] += 1
    assert ((G.cpu().double() - want_G).abs() <= 4 * bound[:, None] + 2.0 ** -8 * want_G.abs()).all()
    assert all(torch.isfinite(x).all() for x in (gh, gw, gb))


@pytest.mark.parametrize("T", [1.0, 2.0])
@pytest.mark.parametrize("banned", BANNED)
@pytest.mark.parametrize("N", [5, 100, 200])
def test_distillation(N, banned, T):
    dev = cuda_or_skip()
    V, K = 1500, 12
    h, w, b = case(N, V, BANNED[banned], 2)
    g = torch.Generator().manual_seed(3)
    allowed = torch.nonzero(torch.isfinite(b))[:, 0]
    ids = allowed[torch.randint(len(allowed), (N, K), generator=g)]
    t = torch.randn(N, K, generator=g) * 3
    z, want_lse, dlse = logit_bounds(h, w, b, T)
    want_loss, _ = ref.distill(h, w, ids, t, b, T)
    size = (z / T).abs().amax(1) + want_lse.abs() + 1 + t.abs().amax(1) / T + math.log(K)
    dloss = T ** 2 * (2 * dlse + 2.0 ** -19 * size)
    d = [x.to(dev) for x in (h, w, ids, t, b)]
    up = torch.ones(N, device=dev)
    for keep in (False, True):
        out = rlk.linear_distill(*d, temperature=T, return_logits=keep)
        loss, lse = out[:2]
        assert ((lse.cpu().double() - want_lse).abs() <= dlse).all()
        assert ((loss.cpu().double() - want_loss).abs() <= dloss).all()
        gh, gw, gb, G = rlk.linear_distill_backward(*d[:4], lse, up, d[4], temperature=T,
                                                    logits=out[2] if keep else None,
                                                    return_grad_logits=True)
        want_G = ref.grad_logits(h, w, ids, t, up.cpu(), b, T)
        assert ((G.cpu().double() - want_G).abs() <= T * 4 * dlse[:, None] + 2.0 ** -8 * want_G.abs()).all()
        assert (G[:, ~torch.isfinite(d[4])] == 0).all()
        assert all(torch.isfinite(x).all() for x in (gh, gw, gb))


@pytest.mark.parametrize("N", [3, 140])
def test_teacher_slots_on_banned_ids(N):
    """A slot that the teacher gives no probability adds nothing; one that it gives some makes the
    divergence infinite."""
    dev = cuda_or_skip()
    h, w, b = case(N, 700, lambda V: slice(64, 96), 4)
    ids = torch.tensor([3, 70, 200]).repeat(N, 1)
    t = torch.tensor([1.0, -1e4, 2.0]).repeat(N, 1)
    d = [x.to(dev) for x in (h, w, ids, t, b)]
    loss, lse = rlk.linear_distill(*d)
    without, _ = rlk.linear_distill(d[0], d[1], d[2][:, ::2], d[3][:, ::2], d[4])
    assert torch.isfinite(loss).all() and (loss - without).abs().max() <= 1e-6 * (1 + without.abs().max())
    d[3][:, 1] = 0.5
    loss, _ = rlk.linear_distill(*d)
    assert (loss == math.inf).all()


@pytest.mark.parametrize("N", [3, 140])
def test_everything_banned_and_rows_of_nan(N):
    dev = cuda_or_skip()
    h, w, b = case(N, 700, lambda V: slice(0, V), 5)
    target = torch.zeros(N, dtype=torch.int64, device=dev)
    _, lse = rlk.linear_logp(h.to(dev), w.to(dev), target, b.to(dev))
    assert (lse == -math.inf).all()
    h, w, b = case(N, 700, lambda V: slice(0, 40), 6)
    clean = rlk.linear_logp(h.to(dev), w.to(dev), target + 50, b.to(dev))
    h[1] = math.nan
    logp, lse = rlk.linear_logp(h.to(dev), w.to(dev), target + 50, b.to(dev))
    assert torch.isnan(logp[1]) and torch.isnan(lse[1])
    rest = torch.arange(N) != 1
    assert bits_equal(logp[rest], clean[0][rest]) and bits_equal(lse[rest], clean[1][rest])
    loss, lse = rlk.linear_distill(h.to(dev), w.to(dev), target[:, None] + 50,
                                   torch.zeros(N, 1, device=dev), b.to(dev))
    assert torch.isnan(loss[1]) and torch.isnan(lse[1])
