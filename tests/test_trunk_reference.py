"""Pins of the trunk's 64-bit definitions: torch's own functions, differences, hand-made blocks."""
import math

import pytest
import torch

import trunk_reference as ref


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_activation_is_torchs_and_its_slope_its_derivative(act):
    g = torch.linspace(-12, 12, 2001, dtype=torch.float64, requires_grad=True)
    own = torch.nn.functional.silu(g) if act == "silu" else \
        torch.nn.functional.gelu(g, approximate="tanh")
    value, slope = ref.activation(g.detach(), act)
    assert torch.allclose(value, own.detach(), rtol=1e-12, atol=1e-14)
    assert torch.allclose(slope, torch.autograd.grad(own.sum(), g)[0], rtol=1e-9, atol=1e-12)
    step = 1e-5
    difference = (ref.activation(g.detach() + step, act)[0] -
                  ref.activation(g.detach() - step, act)[0]) / (2 * step)
    assert torch.allclose(slope, difference, rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_gradient_against_differences(act):
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(5, 7, dtype=torch.float64, generator=gen)
    w = torch.randn(8, 7, dtype=torch.float64, generator=gen)
    d = torch.randn(5, 4, dtype=torch.float64, generator=gen)
    z = x @ w.t()
    G = ref.gated_grad_projections(d, z[:, :4], z[:, 4:], act)
    for grad, at in ((G @ w, x), (G.t() @ x, w)):
        for i in range(0, at.numel(), 3):
            step = torch.zeros_like(at).view(-1)
            step[i] = 1e-6
            step = step.view_as(at)
            up = ref.gated(x + step, w, act) if at is x else ref.gated(x, w + step, act)
            down = ref.gated(x - step, w, act) if at is x else ref.gated(x, w - step, act)
            assert ((up - down) * d).sum() / 2e-6 == pytest.approx(grad.view(-1)[i].item(), rel=1e-6, abs=1e-8)


def test_embedding_gradient_is_autograds():
    gen = torch.Generator().manual_seed(4)
    w = torch.randn(6, 3, dtype=torch.float64, generator=gen, requires_grad=True)
    ids = torch.tensor([2, -1, 5, 2, 6, 0])
    d = torch.randn(6, 3, dtype=torch.float64, generator=gen)
    known = (ids >= 0) & (ids < 6)
    out = w[ids.clamp(0, 5)] * 1.5 * known[:, None]
    assert torch.equal(ref.embedding(ids, w.detach(), 1.5), out.detach())
    want = torch.autograd.grad((out * d).sum(), w)[0]
    assert torch.allclose(ref.embedding_grad(ids, d, 6, 1.5), want, rtol=1e-14, atol=0)
    own_order = ref.embedding_grad_fp32(ids, d.float(), 6, 1.5)
    assert torch.allclose(own_order.double(), want, rtol=1e-6, atol=1e-7)


def test_blocks_by_hand():
    x = torch.zeros(4, 40)
    x[0, :4] = torch.tensor([1.0, -0.5, 127.5 / 64, 0.0078125])      # most 1.99: steps of 2^-6
    x[1, 33] = -3.0
    x[2, 0], x[2, 1], x[2, 39] = math.inf, 1.0, 2.0
    x[3, 39] = math.nan
    q, e = ref.int8_blocks(x)
    assert e.tolist() == [[121, 1], [1, 122], [255, 122], [1, 255]]
    assert q[0, 0, :4].tolist() == [64, -32, 127, 0]                 # 127.5 -> 128, held; 0.5 -> 0
    assert q[1, 1, 1] == -96 and q[2, 1, 7] == 64 and not q[2, 0].any() and not q[3, 1].any()
    back = ref.int8_values(q, e, 40)
    assert back[2, :32].isnan().all() and back[2, 39] == 2 and back[3, 32:].isnan().all()
    assert back[1, 33] == -3 and back[0, 0] == 1


def test_blocks_are_within_half_a_step():
    gen = torch.Generator().manual_seed(5)
    x = (torch.randn(64, 96, generator=gen) * torch.randn(64, 1, generator=gen).exp()).bfloat16()
    q, e = ref.int8_blocks(x)
    back = ref.int8_values(q, e, 96)
    step = ref.power(e - 127).repeat_interleave(32, 1)
    assert ((back - x.double()).abs() <= step / 2).all()
    assert (back.bfloat16().double() == back).all()                  # exact in BF16
