"""What linear_distill_trainable holds between forward and backward, and for how long."""
import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
from helpers import bits_equal, cuda_or_skip

pytestmark = pytest.mark.gpu
N, H, V, K = 512, 64, 40001, 6
LOGITS = 4 * N * 40008


def case(dev, grad=True):
    g = torch.Generator(device=dev).manual_seed(0)
    h = torch.randn(N, H, device=dev, generator=g).bfloat16()
    w = torch.randn(V, H, device=dev, generator=g).bfloat16()
    ids = torch.randint(V, (N, K), device=dev, generator=g)
    t = torch.randn(N, K, device=dev, generator=g)
    return h.requires_grad_(grad), w.requires_grad_(grad), ids, t


def test_logits_are_freed_by_the_backward():
    dev = cuda_or_skip()
    h, w, ids, t = case(dev)
    before = torch.cuda.memory_allocated()
    loss, lse = rlk.linear_distill_trainable(h, w, ids, t)
    assert torch.cuda.memory_allocated() - before >= LOGITS
    loss.sum().backward()
    h.grad = w.grad = None
    assert torch.cuda.memory_allocated() - before < LOGITS // 8     # loss and lse are still held
    with pytest.raises(RuntimeError):
        loss.sum().backward()


def test_copies_are_freed_by_the_backward():
    """Operands that had to be made contiguous are not held past the backward either."""
    dev = cuda_or_skip()
    h, w, ids, t = case(dev, False)
    wt = w.t().contiguous().t().requires_grad_()
    before = torch.cuda.memory_allocated()
    loss, _ = rlk.linear_distill_trainable(h, wt, ids, t, keep_logits=False)
    loss.sum().backward()
    wt.grad = None
    assert torch.cuda.memory_allocated() - before < V * H


def test_logits_are_kept_only_for_a_backward():
    dev = cuda_or_skip()
    h, w, ids, t = case(dev)
    for grad_mode, inputs in ((False, (h, w)), (True, (h.detach(), w.detach()))):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        with torch.set_grad_enabled(grad_mode):
            for keep in (None, True):
                loss, _ = rlk.linear_distill_trainable(*inputs, ids, t, keep_logits=keep)
                assert not loss.requires_grad
        assert torch.cuda.max_memory_allocated() - before < LOGITS


def test_saved_tensor_hooks_see_the_logits():
    dev = cuda_or_skip()
    h, w, ids, t = case(dev)
    loss, _ = rlk.linear_distill_trainable(h, w, ids, t)
    g = torch.randn(N, device=dev)
    want = torch.autograd.grad(loss, (h, w), g)
    packed = []

    def pack(x):
        packed.append(x.numel() * x.element_size())
        return x.cpu()

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda x: x.to(dev)):
        loss, _ = rlk.linear_distill_trainable(h, w, ids, t)
    assert LOGITS in packed
    got = torch.autograd.grad(loss, (h, w), g)
    assert all(bits_equal(a, b) for a, b in zip(got, want))


def test_checkpointing():
    dev = cuda_or_skip()
    from torch.utils.checkpoint import checkpoint
    h, w, ids, t = case(dev)
    g = torch.randn(N, device=dev)
    want = torch.autograd.grad(rlk.linear_distill_trainable(h, w, ids, t)[0], (h, w), g)
    loss = checkpoint(lambda a, b: rlk.linear_distill_trainable(a, b, ids, t)[0], h, w,
                      use_reentrant=False)
    got = torch.autograd.grad(loss, (h, w), g)
    assert all(bits_equal(a, b) for a, b in zip(got, want))


def test_inputs_changed_in_place_are_noticed():
    dev = cuda_or_skip()
    h, w, ids, t = case(dev)
    x = h * 1
    loss, _ = rlk.linear_distill_trainable(x, w, ids, t)
    x.detach().zero_()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.sum().backward()
