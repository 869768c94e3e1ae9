"""The gated block against its definition, and the identities that tie it to det_linear."""
import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
import trunk_reference as ref
from helpers import bits_equal, cuda_or_skip

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
ACTS = ["silu", "gelu_tanh"]

# rows across the loops' limits (32 and 128 rows in the one-CTA loop, 256 in the 2-SM one), odd and
# whole reductions and inner widths, fewer columns than a tile and several tiles
SHAPES = [(1, 1, 1), (1, 64, 128), (2, 8, 31), (17, 65, 33), (31, 200, 300), (32, 128, 129), (33, 63, 127),
          (64, 256, 1024), (127, 100, 40), (128, 72, 257), (129, 64, 128), (200, 1000, 130), (256, 320, 96),
          (257, 128, 385), (300, 65, 1000), (513, 192, 64),
          (300, 4000, 600),        # both products of the backward in one launch
          (2600, 64, 7100)]        # tiles handed out from the workspace's counter


def operands(M, K, F, seed=0, loud=1.0):
    g = torch.Generator().manual_seed(1000 * M + 10 * K + F + seed)
    dev = cuda_or_skip()
    x = torch.randn(M, K, generator=g).to(BF16).to(dev)
    w = (torch.randn(2 * F, K, generator=g) * (loud / K ** 0.5)).to(BF16).to(dev)
    d = torch.randn(M, F, generator=g).to(BF16).to(dev)
    return x, w, d


def projections(x, w):
    z = rlk.det_linear(x, w, FP32)
    f = w.size(0) // 2
    return z[:, :f], z[:, f:]


def argument_bound(g, act):
    """Relative error of sigmoid(a) and of sigmoid(-a) in FP32: the argument a(g) of FP32 g is off by at
    most 4 roundings and its product with log2(e) by 2 more (6 |a| 2^-24 of the exponential), 2^x by
    2^-22, the sum, the reciprocal (2^-23) and the products by 2^-22 together."""
    return (3 * ref.argument(g.double(), act)[0].abs() + 8) * 2.0 ** -23


def value_bound(g, u, act, dtype):
    h = ref.activation(g.double(), act)[0] * u.double()
    return h, h.abs() * argument_bound(g, act) + h.abs() * (torch.finfo(dtype).eps / 2 + 2.0 ** -23) + 1e-36


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,K,F", SHAPES)
def test_forward(M, K, F, act):
    x, w, _ = operands(M, K, F, loud=2.0)
    g, u = projections(x, w)
    for dtype in (BF16, FP32):
        h = rlk.gated_linear(x, w, act, dtype)
        assert h.dtype == dtype and h.shape == (M, F)
        want, bound = value_bound(g, u, act, dtype)
        assert ((h.double() - want).abs() <= bound).all()
    # the whole block: FP32 sums of K products
    want = ref.gated(x, w, act)
    assert (h.double() - want).norm() <= 1e-5 * want.norm()
    assert rlk.device_error() == 0


@pytest.mark.parametrize("act", ACTS)
def test_forward_over_the_range_of_the_activation(act):
    # one product a projection: g is the weight's number times one, u is one
    dev = cuda_or_skip()
    values = torch.cat([torch.linspace(-100, 100, 2001), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e10, -1e10, 3e38, -3e38])])
    F = values.numel()
    w = torch.zeros(2 * F, 8)
    w[:F, 0], w[F:, 1] = values, 1.0
    x = torch.zeros(3, 8)
    x[:, :2] = 1.0
    x, w = x.to(BF16).to(dev), w.to(BF16).to(dev)
    g, u = projections(x, w)
    h = rlk.gated_linear(x, w, act, FP32)
    want, bound = value_bound(g, u, act, FP32)
    assert ((h.double() - want).abs() <= bound + 1e-35).all() and torch.isfinite(h).all()
    d = torch.ones(3, F, device=dev)
    G = rlk.gated_linear_backward(d, x, w, act, return_grad_projections=True)[2]
    check_grad_projections(G, d, g, u, act)
    assert torch.isfinite(G).all()


def check_grad_projections(G, d, g, u, act):
    F = g.size(1)
    want = ref.gated_grad_projections(d, g, u, act)
    a, da = ref.argument(g.double(), act)
    s, rest = torch.sigmoid(a), torch.sigmoid(-a)
    off = argument_bound(g, act) + 2.0 ** -21
    parts = s + (g.double() * s * rest * da).abs() * 3            # three factors, each off by `off`
    bound = torch.cat([(d.double() * u.double()).abs() * parts * off, (d.double() * g.double() * s).abs() * off], 1)
    bound = bound + (want.abs() + bound) * 2.0 ** -8 + 1e-30      # BF16's half step
    assert G.shape == (g.size(0), 2 * F)
    assert ((G.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,K,F", SHAPES)
def test_backward(M, K, F, act):
    x, w, d = operands(M, K, F, 1, loud=2.0)
    g, u = projections(x, w)
    for grad in (d, d.float() * 1.001):
        gx, gw, G = rlk.gated_linear_backward(grad, x, w, act, return_grad_projections=True)
        check_grad_projections(G, grad, g, u, act)
        # the products are det_linear's, bit for bit
        want_x, want_w = rlk.det_linear_backward(G.contiguous(), x, w)
        assert bits_equal(gx, want_x) and bits_equal(gw, want_w)
    assert rlk.device_error() == 0


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,K,F", SHAPES)
def test_kept_projections(M, K, F, act):
    x, w, d = operands(M, K, F, 2, loud=2.0)
    g, u = projections(x, w)
    h = rlk.gated_linear(x, w, act)
    h32, kept = rlk.gated_linear(x, w, act, keep="fp32")
    h8, (q, e) = rlk.gated_linear(x, w, act, keep="int8")
    assert bits_equal(h, h32) and bits_equal(h, h8)
    assert bits_equal(kept[:, 0, :F] + 0.0, g + 0.0) and bits_equal(kept[:, 1, :F] + 0.0, u + 0.0)
    assert not kept[:, :, F:].any() and not q[:, :, F:].any()
    for plane, z in ((0, g), (1, u)):
        want_q, want_e = rlk.pack_int8(z)
        assert torch.equal(q[:, plane, :F], want_q) and torch.equal(e[:, plane], want_e)
    # from FP32 the same bits as forming them again; from 8 bits the gradient at the stored values
    for grad in (d, d.float() * 1.001):
        again = rlk.gated_linear_backward(grad, x, w, act, return_grad_projections=True)
        held = rlk.gated_linear_backward(grad, x, w, act, kept=kept, return_grad_projections=True)
        assert all(bits_equal(a, b) for a, b in zip(again, held))
        gx, gw, G = rlk.gated_linear_backward(grad, x, w, act, kept=(q, e), return_grad_projections=True)
        stored = [rlk.unpack_int8(q[:, i, :F], e[:, i], FP32) for i in (0, 1)]
        check_grad_projections(G, grad, *stored, act)
        want_x, want_w = rlk.det_linear_backward(G.contiguous(), x, w)
        assert bits_equal(gx, want_x) and bits_equal(gw, want_w)
    assert rlk.device_error() == 0


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("K,F", [(200, 300), (64, 1024), (1000, 70)])
def test_rows_do_not_depend_on_the_batch(K, F, act):
    x, w, d = operands(700, K, F, 3)
    h, kept = rlk.gated_linear(x, w, act, keep="fp32")
    gx = rlk.gated_linear_backward(d, x, w, act, grad_w=False)[0]
    for a, b in ((0, 1), (5, 22), (100, 228), (100, 229), (300, 556), (699, 700), (0, 600)):
        part, part_kept = rlk.gated_linear(x[a:b], w, act, keep="fp32")
        assert bits_equal(part, h[a:b]) and bits_equal(part_kept, kept[a:b])
        one, none = rlk.gated_linear_backward(d[a:b], x[a:b], w, act, grad_w=False)
        assert none is None and bits_equal(one, gx[a:b])
    assert bits_equal(rlk.gated_linear(x, w, act), h)


@pytest.mark.parametrize("M", [9, 100, 300])
def test_any_layout(M):
    K, F = 100, 70
    x, w, d = operands(M, K, F, 4)
    h, kept = rlk.gated_linear(x, w, keep="int8")
    grads = rlk.gated_linear_backward(d, x, w)
    held = rlk.gated_linear_backward(d, x, w, kept=kept)
    for px, pw, pd, off in ((104, 104, 72, 0), (101, 103, 71, 1), (112, 112, 80, 8), (104, 104, 72, 4)):
        def wide(t, pitch):
            buf = torch.full((t.size(0) * pitch + off,), float("nan"), dtype=t.dtype, device=t.device)
            return buf[off:].view(t.size(0), pitch)[:, :t.size(1)].copy_(t)
        vx, vw, vd = wide(x, px), wide(w, pw), wide(d, pd)
        hv, kv = rlk.gated_linear(vx, vw, keep="int8")
        assert bits_equal(hv, h) and all(torch.equal(a, b) for a, b in zip(kv, kept))
        assert all(bits_equal(a, b) for a, b in zip(rlk.gated_linear_backward(vd, vx, vw), grads))
        assert all(bits_equal(a, b) for a, b in zip(rlk.gated_linear_backward(vd, vx, vw, kept=kept), held))
    if M == 300:
        x3, d3 = x.view(3, 100, K), d.view(3, 100, F)
        assert bits_equal(rlk.gated_linear(x3, w), h.view(3, 100, F))
        g3 = rlk.gated_linear_backward(d3, x3, w)
        assert g3[0].shape == x3.shape and bits_equal(g3[0].view(M, K), grads[0]) and bits_equal(g3[1], grads[1])
    assert bits_equal(rlk.gated_linear(x.t().contiguous().t(), w), h)
    # one row without leading dimensions; a gradient that is one number
    assert bits_equal(rlk.gated_linear(x[3], w), h[3])
    alone = rlk.gated_linear_backward(d[3], x[3], w)
    assert bits_equal(alone[0], grads[0][3]) and alone[1].shape == w.shape
    ones = rlk.gated_linear_backward(torch.ones_like(d), x, w)
    same = rlk.gated_linear_backward(torch.ones((), dtype=BF16, device=d.device).expand(M, F), x, w)
    assert all(bits_equal(a, b) for a, b in zip(ones, same))


def test_not_finite_numbers_stay_in_their_rows():
    x, w, d = operands(140, 64, 96, 5)
    h, kept = rlk.gated_linear(x, w, keep="int8")
    for rows in (slice(0, 20), slice(0, 140)):
        y = x[rows].clone()
        y[7, 3], y[11, 0] = float("nan"), float("inf")
        got, (q, e) = rlk.gated_linear(y, w, keep="int8")
        fine = torch.ones(y.size(0), dtype=torch.bool, device=y.device)
        fine[[7, 11]] = False
        assert bits_equal(got[fine], h[rows][fine]) and torch.equal(q[fine], kept[0][rows][fine])
        assert got[7].isnan().all() and (e[[7, 11]] == 255).all()
        gx = rlk.gated_linear_backward(d[rows], y, w, kept=(q, e), grad_w=False)[0]
        assert gx[[7, 11]].isnan().all() and torch.isfinite(gx[fine]).all()


@pytest.mark.parametrize("checkpoint", [None, "fp32", "int8", "again"])
@pytest.mark.parametrize("act", ACTS)
def test_trainable(act, checkpoint):
    x, w, d = operands(150, 96, 100, 6)
    x3 = x.view(3, 50, 96).requires_grad_()
    w.requires_grad_()
    d3 = d.view(3, 50, 100)
    h = rlk.gated_linear_trainable(x3, w, act, checkpoint=checkpoint)
    assert bits_equal(h, rlk.gated_linear(x3.detach(), w.detach(), act))
    gx, gw = torch.autograd.grad(h, (x3, w), d3)
    xd, wd = x.detach(), w.detach()
    if checkpoint == "int8":
        _, kept = rlk.gated_linear(xd, wd, act, keep="int8")
        want = rlk.gated_linear_backward(d, rlk.unpack_int8(*rlk.pack_int8(xd)), wd, act, kept=kept)
    else:
        want = rlk.gated_linear_backward(d, xd, wd, act)
    assert gx.shape == x3.shape and bits_equal(gx.view(150, 96), want[0]) and bits_equal(gw, want[1])
    only_x, = torch.autograd.grad(rlk.gated_linear_trainable(x3, wd, act, checkpoint=checkpoint), x3, d3)
    only_w, = torch.autograd.grad(rlk.gated_linear_trainable(x3.detach(), w, act, checkpoint=checkpoint), w, d3)
    assert bits_equal(only_x, gx) and bits_equal(only_w, gw)
    # against the 64-bit gradient: G and the result are rounded to BF16, each at most 2^-8 relative
    # (8 bits: a value is off by at most 2^-7 of its block's largest, here some 3 root mean squares)
    g, u = (xd.double() @ wd[:100].double().t(), xd.double() @ wd[100:].double().t())
    G = ref.gated_grad_projections(d, g, u, act)
    for got, exact in ((gx.view(150, 96), G @ wd.double()), (gw, G.t() @ xd.double())):
        off = (got.double() - exact).norm() / exact.norm()
        assert off <= (4 * 3 * 2.0 ** -7 if checkpoint == "int8" else 2 * 2.0 ** -8)


def test_what_is_held():
    x, w, _ = operands(64, 96, 100, 7)
    x.requires_grad_()
    w.requires_grad_()
    sizes = {"fp32": 64 * 2 * 128 * 4, "int8": 64 * (2 * 128 + 2 * 4 + 96 + 3), "again": 0}
    for checkpoint, size in sizes.items():
        held = []
        with torch.autograd.graph.saved_tensors_hooks(lambda t: held.append(t) or t, lambda t: t):
            rlk.gated_linear_trainable(x, w, checkpoint=checkpoint)
        mine = [t for t in held if t.data_ptr() not in (x.data_ptr(), w.data_ptr())]
        assert sum(t.numel() * t.element_size() for t in mine) == size, checkpoint
        assert (checkpoint == "int8") == all(t.data_ptr() != x.data_ptr() for t in held)


def test_empty_and_refusals():
    x, w, d = operands(4, 16, 24, 8)
    assert rlk.gated_linear(x[:0], w).shape == (0, 24)
    gx, gw = rlk.gated_linear_backward(d[:0], x[:0], w)
    assert gx.shape == (0, 16) and gw.shape == (48, 16) and not gw.any()
    h, kept = rlk.gated_linear(x[:0], w, keep="int8")
    assert kept[0].shape == (0, 2, 32) and kept[1].shape == (0, 2, 1)
    with pytest.raises(ValueError, match="activation"):
        rlk.gated_linear(x, w, "relu")
    with pytest.raises(ValueError, match="keep"):
        rlk.gated_linear(x, w, keep="bf16")
    with pytest.raises(ValueError, match="2 F"):
        rlk.gated_linear(x, w[:47])
    with pytest.raises(TypeError):
        rlk.gated_linear(x.float(), w)
    with pytest.raises(ValueError, match="dH"):
        rlk.gated_linear_backward(d[:, :23], x, w)
    _, kept = rlk.gated_linear(x, w, keep="int8")
    for bad in (kept[0], kept[0].float()[:3], (kept[0][:3], kept[1][:3]), (kept[0], kept[1].int()),
                (kept[0].float(), kept[1])):
        with pytest.raises(ValueError, match="kept"):
            rlk.gated_linear_backward(d, x, w, kept=bad)
    with pytest.raises(ValueError, match="dX or dW"):
        rlk.gated_linear_backward(d, x, w, grad_x=False, grad_w=False, return_grad_projections=True)
    with pytest.raises(ValueError, match="checkpoint"):
        rlk.gated_linear_trainable(x, w, checkpoint="bf16")
    with pytest.raises(RuntimeError, match="forward-only"):
        rlk.gated_linear(x.requires_grad_(), w)
