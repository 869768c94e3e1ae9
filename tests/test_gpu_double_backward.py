"""The gradients have no derivatives of their own: asking for one is an error, not a zero."""
import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
from helpers import cuda_or_skip

pytestmark = pytest.mark.gpu


def calls(dev):
    g = torch.Generator(device=dev).manual_seed(0)
    x = torch.randn(20, 32, device=dev, generator=g).bfloat16().requires_grad_()
    w = torch.randn(300, 32, device=dev, generator=g).bfloat16().requires_grad_()
    ids = torch.randint(300, (20, 3), device=dev, generator=g)
    t = torch.randn(20, 3, device=dev, generator=g)
    return x, w, {
        "linear_logp": lambda: rlk.linear_logp_trainable(x, w, ids[:, 0].contiguous())[0],
        "linear_distill": lambda: rlk.linear_distill_trainable(x, w, ids, t)[0],
        "det_gemm": lambda: rlk.det_gemm_trainable(x, w.t()),
        "det_linear": lambda: rlk.det_linear_trainable(x, w),
    }


@pytest.mark.parametrize("name", ["linear_logp", "linear_distill", "det_gemm", "det_linear"])
def test_second_derivative_is_refused(name):
    dev = cuda_or_skip()
    x, w, of = calls(dev)
    out = of[name]()
    g = torch.ones_like(out).requires_grad_()
    gx, = torch.autograd.grad(out, (x,), g, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        gx.float().square().sum().backward()
