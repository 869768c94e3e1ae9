"""Activations in 8 bits against their 64-bit definition: whole numbers, so equality throughout."""
import math

import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
import trunk_reference as ref
from helpers import bits_equal, cuda_or_skip

pytestmark = pytest.mark.gpu


def rows_of(rows, cols, dtype, seed=0, pitch=None, offset=0):
    """Rows of widely spread sizes, some columns loud; in a wider, shifted buffer if asked."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * (4 * torch.randn(rows, 1, generator=g)).exp()
    x[:, torch.randint(cols, (1 + cols // 50,), generator=g)] *= 9
    x = x.to(dtype).to(cuda_or_skip())
    if pitch is None:
        return x
    wide = torch.zeros(rows * pitch + offset, dtype=dtype, device=x.device)
    out = wide[offset:offset + rows * pitch].view(rows, pitch)[:, :cols]
    return out.copy_(x)


def check(x):
    q, e = rlk.pack_int8(x)
    want_q, want_e = ref.int8_blocks(x.float())
    assert q.dtype == torch.int8 and e.dtype == torch.uint8
    assert torch.equal(e.long(), want_e)
    assert torch.equal(q.long(), want_q.flatten(1)[:, :x.size(1)])
    want = ref.int8_values(want_q, want_e, x.size(1))
    for dtype in (torch.bfloat16, torch.float32):
        back = rlk.unpack_int8(q, e, dtype)
        assert torch.equal(back.double().nan_to_num(7.7), want.nan_to_num(7.7))
    assert rlk.device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (3, 32), (2, 33), (65, 64), (7, 100), (300, 255),
                                       (129, 1000), (17, 2047), (33, 2049), (5, 4104), (2, 20001)])
def test_against_the_definition(rows, cols, dtype):
    check(rows_of(rows, cols, dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pitch,offset", [(101, 0), (104, 0), (104, 1), (112, 8), (120, 3)])
def test_any_pitch_and_offset(dtype, pitch, offset):
    check(rows_of(37, 100, dtype, 1, pitch, offset))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_extremes(dtype):
    x = rows_of(12, 70, dtype, 2)
    x[0] = 0
    x[1, 3] = math.nan
    x[2, 40], x[3, 69] = math.inf, -math.inf
    x[4] = 1e-38
    x[5] = 1e-40 if dtype == torch.float32 else 1e-39
    x[6] = torch.finfo(dtype).max
    x[7] = -torch.finfo(dtype).max
    x[8, :32] = torch.tensor([2.0 ** -i for i in range(32)])
    x[9, :4] = torch.tensor([127.5, 63.5, 0.5, -0.5])            # halves of a step: to even
    x[9, 4:32] = 0
    x[10, :2] = torch.tensor([255.0, -254.5])                     # held to 127 steps of 2
    x[11] = -0.0
    check(x)


def test_leading_dimensions_strides_and_empty():
    x = rows_of(60, 48, torch.bfloat16, 3)
    q, e = rlk.pack_int8(x)
    q3, e3 = rlk.pack_int8(x.view(3, 4, 5, 48))
    assert q3.shape == (3, 4, 5, 48) and e3.shape == (3, 4, 5, 2)
    assert torch.equal(q3.reshape(60, 48), q) and torch.equal(e3.reshape(60, 2), e)
    back = rlk.unpack_int8(q, e)
    assert torch.equal(rlk.unpack_int8(q3, e3).view(60, 48), back)
    # values that are not rows of whole blocks are copied into such rows
    assert torch.equal(rlk.unpack_int8(q.contiguous(), e), back)
    assert torch.equal(rlk.unpack_int8(q.t().contiguous().t(), e.t().contiguous().t()), back)
    one = rlk.pack_int8(x[7])
    assert one[0].shape == (48,) and torch.equal(rlk.unpack_int8(*one), back[7])
    assert torch.equal(rlk.pack_int8(x.t().contiguous().t())[0], q)
    q0, e0 = rlk.pack_int8(x[:0])
    assert q0.shape == (0, 48) and rlk.unpack_int8(q0, e0).shape == (0, 48)


def test_rows_do_not_depend_on_each_other():
    x = rows_of(200, 333, torch.float32, 4)
    q, e = rlk.pack_int8(x)
    for a, b in ((0, 1), (17, 80), (199, 200)):
        qa, ea = rlk.pack_int8(x[a:b])
        assert torch.equal(qa, q[a:b]) and torch.equal(ea, e[a:b])
    assert bits_equal(rlk.unpack_int8(q, e)[17:80], rlk.unpack_int8(q[17:80], e[17:80]))


def test_linear_with_a_checkpoint():
    g = torch.Generator().manual_seed(6)
    dev = cuda_or_skip()
    x = torch.randn(3, 50, 100, generator=g).to(dev).bfloat16().requires_grad_()
    w = torch.randn(70, 100, generator=g).to(dev).bfloat16().requires_grad_()
    d = torch.randn(3, 50, 70, generator=g).to(dev).bfloat16()
    y = rlk.det_linear_trainable(x, w, checkpoint="int8")
    plain = rlk.det_linear_trainable(x, w)
    assert bits_equal(y, plain)
    gx, gw = torch.autograd.grad(y, (x, w), d)
    held = rlk.unpack_int8(*rlk.pack_int8(x.detach()))
    want_x, want_w = rlk.det_linear_backward(d, held, w.detach())
    assert gx.shape == x.shape and bits_equal(gx, want_x.view_as(x)) and bits_equal(gw, want_w)
    assert bits_equal(gx, torch.autograd.grad(plain, x, d)[0])
    # a gradient of one of them alone
    assert bits_equal(torch.autograd.grad(rlk.det_linear_trainable(x, w.detach(), checkpoint="int8"), x, d)[0], gx)
    assert bits_equal(torch.autograd.grad(rlk.det_linear_trainable(x.detach(), w, checkpoint="int8"), w, d)[0], gw)
    # what is held: a byte a value and one in 32
    held = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: held.append(t) or t, lambda t: t):
        rlk.det_linear_trainable(x, w, checkpoint="int8")
    assert sum(t.untyped_storage().nbytes() for t in held if t.data_ptr() != w.data_ptr()) == 150 * 128 + 150 * 4


def test_refusals():
    x = rows_of(4, 64, torch.bfloat16)
    q, e = rlk.pack_int8(x)
    with pytest.raises(TypeError):
        rlk.pack_int8(x.half())
    with pytest.raises(TypeError):
        rlk.unpack_int8(q.to(torch.uint8), e)
    with pytest.raises(ValueError):
        rlk.unpack_int8(q, e[:, :1])
    with pytest.raises(ValueError):
        rlk.det_linear_trainable(x, x, checkpoint="fp8")
