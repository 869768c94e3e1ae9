"""The gated block with a weight that needs no gradient: nothing is held or allocated for a product
that is not formed."""
import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
from helpers import bits_equal, cuda_or_skip

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
ROWS, K, F = 2048, 4096, 64              # X is 16 MB, the projections' gradient 0.5 MB
SLACK = 2 << 20                          # the allocator's rounding of each of a few tensors


def operands(pitch=K):
    dev = cuda_or_skip()
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn(ROWS, pitch, device=dev, generator=g).to(BF16)[:, :K]
    w = (torch.randn(2 * F, pitch, device=dev, generator=g) / K ** 0.5).to(BF16)[:, :K]
    d = torch.randn(ROWS, F, device=dev, generator=g).to(BF16)
    return x, w, d


def peak(call):
    """What call returns, and the most bytes that were allocated on the way beyond those before it."""
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out = call()
    torch.cuda.synchronize()
    return out, torch.cuda.max_memory_allocated() - before


@pytest.mark.parametrize("checkpoint", ["fp32", "int8", "again"])
def test_the_input_is_not_held(checkpoint):
    x, w, _ = operands()
    x.requires_grad_()
    held = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: held.append(t) or t, lambda t: t):
        rlk.gated_linear_trainable(x, w, checkpoint=checkpoint)
    assert any(t.data_ptr() == x.data_ptr() for t in held) == (checkpoint == "again")
    kept = {"fp32": ROWS * 2 * F * 4, "int8": ROWS * (2 * F + 2 * F // 32), "again": 0}[checkpoint]
    assert sum(t.numel() * t.element_size() for t in held
               if t.data_ptr() not in (x.data_ptr(), w.data_ptr())) == kept


@pytest.mark.parametrize("shape", [(ROWS,), (2, ROWS // 2)])
@pytest.mark.parametrize("checkpoint", ["fp32", "int8"])
def test_memory_of_the_backward(checkpoint, shape):
    x, w, d = operands()
    x, d = x.view(*shape, K).requires_grad_(), d.view(*shape, F)
    h = rlk.gated_linear_trainable(x, w, checkpoint=checkpoint)
    (gx,), most = peak(lambda: torch.autograd.grad(h, x, d))
    # the gradient and the projections' gradient in the workspace
    assert most <= ROWS * K * 2 + ROWS * 2 * F * 2 + SLACK
    kept = rlk.gated_linear(x.detach(), w, keep=checkpoint)[1]
    want = rlk.gated_linear_backward(d, x.detach(), w, kept=kept, grad_w=False)[0]
    assert gx.shape == x.shape and bits_equal(gx, want)


def test_workspace_of_operands_that_are_not_read():
    """An odd pitch asks for a padded copy, but only of an operand that a product reads."""
    x, w, d = operands(K + 1)
    kept = rlk.gated_linear(x, w, keep="int8")[1]
    both = rlk.gated_linear_backward(d, x, w, kept=kept)
    gx, most = peak(lambda: rlk.gated_linear_backward(d, x, w, kept=kept, grad_w=False)[0])
    assert bits_equal(gx, both[0]) and most <= ROWS * K * 2 + ROWS * 2 * F * 2 + 2 * F * K * 2 + SLACK
    gw, most = peak(lambda: rlk.gated_linear_backward(d, x, w, kept=kept, grad_x=False)[1])
    assert bits_equal(gw, both[1]) and most <= 2 * F * K * 2 + ROWS * 2 * F * 2 + ROWS * K * 2 + SLACK
    none, _ = peak(lambda: rlk.gated_linear_backward(d, None, w, kept=kept, grad_w=False))
    assert bits_equal(none[0], both[0]) and none[1] is None


def test_a_missing_input_is_refused_where_it_is_read():
    x, w, d = operands()
    kept = rlk.gated_linear(x, w, keep="fp32")[1]
    for named in (dict(kept=kept), dict(grad_w=False)):
        with pytest.raises(ValueError, match="X"):
            rlk.gated_linear_backward(d, None, w, **named)
    with pytest.raises(ValueError, match="kept"):
        rlk.gated_linear_backward(d[:5], None, w, kept=kept, grad_w=False)
    with pytest.raises(ValueError, match="dH"):
        rlk.gated_linear_backward(d[:, :5], None, w, kept=kept, grad_w=False)
