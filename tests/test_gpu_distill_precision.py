"""The distillation loss where its parts nearly cancel: students close to the teacher, at
temperatures that multiply the loss by T^2.  Logits are small multiples of 1/8, exact in FP32, so what
is measured is the loss itself."""
import math

import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
import distill_reference as ref
from helpers import cuda_or_skip

pytestmark = pytest.mark.gpu


def case(N, V, seed, noise):
    """hidden [N, 8], weight [V, 8], every id as a slot, teacher logits near the student's."""
    g = torch.Generator().manual_seed(seed)
    h = torch.randint(-6, 7, (N, 8), generator=g).float()
    w = torch.randint(-4, 5, (V, 8), generator=g).float() / 16
    z = h @ w.T
    t = z + torch.randn(N, V, generator=g) * noise
    return h.bfloat16(), w.bfloat16(), torch.arange(V).repeat(N, 1), t


def bound(h, w, ids, t, T, tl=None):
    """T^2 Q times the relative errors of the student's sum of exponentials (2^-22 of each, as much of
    their sums, 2^-23 of the exponents), of the teacher's (2^-23) and, against log q - log p, of q
    (2^-22); T times the FP32 sum of q z; one rounding of the loss."""
    z = h.double() @ w.double().T
    logp = torch.log_softmax(z / T, 1)
    used, logq, q = ref.teacher(ids, t, w.size(0), T, tl)
    terms = torch.where(used, logq - logp.gather(1, ids), 0.0).abs().amax(1)
    Q, size = q.sum(1), z.abs().amax(1)
    loss, _ = ref.distill(h, w, ids, t, None, T, tl)
    return Q * (T ** 2 * (2.0 ** -21 + 2.0 ** -23 + 2.0 ** -22 * terms) + T * 2.0 ** -22 * size +
                T * 2.0 ** -21 * size) + 2.0 ** -23 * loss.abs()


@pytest.mark.parametrize("T", [1.0, 2.0, 10.0, 100.0])
@pytest.mark.parametrize("noise", [0.0, 0.01, 1.0])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("N", [100, 300])
def test_students_close_to_the_teacher(N, tail, noise, T):
    dev = cuda_or_skip()
    h, w, ids, t = case(N, 1000, 1, noise)
    tl = torch.logsumexp(t.double() / T, 1).float() if tail else None
    want, want_lse = ref.distill(h, w, ids, t, None, T, tl)
    d = [x.to(dev) for x in (h, w, ids, t)]
    loss, lse = rlk.linear_distill(*d, temperature=T, teacher_lse=None if tl is None else tl.to(dev))
    error = (loss.cpu().double() - want).abs()
    assert (error <= bound(h, w, ids, t, T, tl)).all(), (error / bound(h, w, ids, t, T, tl)).max()
    assert ((lse.cpu().double() - want_lse).abs() <= 2.0 ** -21 + 2.0 ** -23 * want_lse.abs()).all()


def test_infinite_teacher_logits_are_not_hidden():
    """A used slot's +inf makes the loss NaN, with the teacher's own log-sum-exp too."""
    dev = cuda_or_skip()
    h, w, ids, t = case(40, 300, 2, 1.0)
    tl = torch.logsumexp(t, 1)
    t[7, 5], t[9, 200] = math.inf, math.nan
    d = [x.to(dev) for x in (h, w, ids, t, tl)]
    for lse in (None, d[4]):
        loss, _ = rlk.linear_distill(*d[:4], teacher_lse=lse)
        bad = torch.isnan(loss)
        assert bad[7] and bad[9] and bad.sum() == 2
