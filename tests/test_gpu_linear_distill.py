"""Distillation from a teacher's top logits on the GPU: the loss, log-sum-exp and gradients
against 64 bits, bit for bit against the linear-logp operators where they coincide, and
what must not change a bit."""
import math

import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
import distill_reference as ref
from helpers import GEMM_FP32_REL_FRO, bits_equal, cuda_or_skip

pytestmark = pytest.mark.gpu


def inputs(N, H, V, K, seed=0, bias=False, dtype=torch.float32, scale=2.0, tail=False, T=1.0):
    """CPU tensors: hidden, weight, ids, teacher logits, bias, teacher lse."""
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(N, H, generator=g).bfloat16()
    w = (torch.randn(V, H, generator=g) * (scale / math.sqrt(H))).bfloat16()
    b = torch.randn(V, generator=g) * 0.1 if bias else None
    ids = torch.randint(V, (N, K), generator=g)        # repeats happen
    t = (torch.randn(N, K, generator=g) * 3).to(dtype)
    lse = torch.logsumexp(t.float() / T, 1) + 0.2 if tail and K else None
    return h, w, ids, t, b, lse


def on(dev, *ts):
    return [None if t is None else t.to(dev) for t in ts]


def check_forward(dev, h, w, ids, t, b, lse, T):
    hd, wd, idd, td, bd, ld = on(dev, h, w, ids, t, b, lse)
    loss, got = rlk.linear_distill(hd, wd, idd, td, bd, temperature=T, teacher_lse=ld)
    assert rlk.device_error() == 0
    want_loss, want_lse = ref.distill(h, w, ids, t, b, T, lse)
    dloss, dlse, _ = ref.bounds(h, w, ids, t, b, T, lse)
    e_lse = (got.cpu().double() - want_lse).abs()
    e_loss = (loss.cpu().double() - want_loss).abs()
    assert (e_lse <= dlse).all(), (e_lse - dlse).max()
    assert (e_loss <= dloss).all(), (e_loss / dloss).max()
    return loss, got


SHAPES = [  # N, H, V, K
    (1, 1, 1, 1), (1, 8, 2, 2), (3, 33, 33, 5), (17, 128, 1000, 64), (32, 64, 257, 1),
    (33, 72, 511, 7), (128, 256, 1024, 8), (129, 64, 999, 33), (257, 40, 513, 100),
    (300, 512, 4099, 65), (5, 16, 263000, 129), (2, 24, 1500, 1024),
]


@pytest.mark.parametrize("N,H,V,K", SHAPES)
@pytest.mark.parametrize("T,bias,dtype,tail", [(1.0, False, torch.float32, False),
                                               (2.0, True, torch.bfloat16, True)])
def test_forward(N, H, V, K, T, bias, dtype, tail):
    dev = cuda_or_skip()
    check_forward(dev, *inputs(N, H, V, K, 1, bias, dtype, tail=tail, T=T), T)


@pytest.mark.parametrize("N", [20, 200])
def test_empty_slots(N):
    """Padding by id and by logit, ids past the vocabulary, rows without any slot, and what the
    empty slots' logits hold."""
    dev = cuda_or_skip()
    h, w, ids, t, b, _ = inputs(N, 96, 700, 12, 2, True)
    ids[0::5, 3:] = -1
    t[0::5, 3] = math.nan
    t[0::5, 4] = math.inf
    t[1::5, ::2] = -math.inf
    ids[2::5, 1] = 700
    ids[2::5, 2] = 1 << 40
    ids[3::5] = -1
    t[4::5] = -math.inf
    loss, _ = check_forward(dev, h, w, ids, t.where(torch.isfinite(t) | (t == -math.inf), 0.0), b,
                            None, 1.0)
    hd, wd, idd, td, bd = on(dev, h, w, ids, t, b)
    again, lse = rlk.linear_distill(hd, wd, idd, td, bd)
    assert bits_equal(again, loss)
    assert (loss[3::5] == 0).all() and (loss[4::5] == 0).all() and (loss[0::5] != 0).all()
    g = torch.ones(N, device=dev)
    gh, _, _, G = rlk.linear_distill_backward(hd, wd, idd, td, lse, g, bd, return_grad_logits=True)
    assert (G[3::5] == 0).all() and (G[4::5] == 0).all() and (gh[3::5] == 0).all()
    assert torch.isfinite(G).all()
    # a used slot's NaN or infinity is not hidden
    td[0, 0], td[1, 1] = math.nan, math.inf
    bad, _ = rlk.linear_distill(hd, wd, idd, td, bd)
    assert torch.isnan(bad[:2]).all() and bits_equal(bad[2:], loss[2:])


def test_no_slots_and_no_rows():
    dev = cuda_or_skip()
    h, w, ids, t, b, _ = on(dev, *inputs(6, 32, 300, 4, 3, True))
    loss, lse = rlk.linear_distill(h, w, ids[:, :0], t[:, :0], b)
    assert (loss == 0).all()
    assert bits_equal(lse, rlk.linear_logp(h, w, torch.zeros(6, dtype=torch.int64, device=dev), b)[1])
    gh, gw, gb = rlk.linear_distill_backward(h, w, ids[:, :0], t[:, :0], lse, torch.ones_like(loss), b)
    assert not gh.any() and not gw.any() and not gb.any()
    loss, lse = rlk.linear_distill(h[:0], w, ids[:0], t[:0], b)
    assert loss.shape == (0,) and lse.shape == (0,)
    gh, gw, gb = rlk.linear_distill_backward(h[:0], w, ids[:0], t[:0], lse, loss, b)
    assert gh.shape == (0, 32) and not gw.any() and not gb.any()


@pytest.mark.parametrize("N,H,V,K,T,bias,tail", [
    (1, 1, 1, 1, 1.0, False, False), (3, 33, 33, 5, 1.0, True, True), (40, 64, 300, 17, 2.0, True, False),
    (130, 128, 1000, 64, 1.0, False, True), (300, 96, 519, 33, 0.5, True, False),
    (513, 72, 2050, 9, 1.5, True, True)])
def test_backward(N, H, V, K, T, bias, tail):
    dev = cuda_or_skip()
    h, w, ids, t, b, tl = inputs(N, H, V, K, 4, bias, tail=tail, T=T)
    ids[::7, K // 2:] = -1
    g = torch.randn(N, generator=torch.Generator().manual_seed(5))
    hd, wd, idd, td, bd, tld, gd = on(dev, h, w, ids, t, b, tl, g)
    _, lse = rlk.linear_distill(hd, wd, idd, td, bd, temperature=T, teacher_lse=tld)
    gh, gw, gb, G = rlk.linear_distill_backward(hd, wd, idd, td, lse, gd, bd, temperature=T,
                                                teacher_lse=tld, out_dtype=torch.float32,
                                                return_grad_logits=True)
    assert rlk.device_error() == 0
    G = G.cpu().double()
    want = ref.grad_logits(h, w, ids, t, g, b, T, tl)
    # G: the error of p, of the K-slot q's (FP32 exponentials of sums) and one BF16 rounding
    _, _, dp = ref.bounds(h, w, ids, t, b, T, tl)
    used, _, q = ref.teacher(ids, t, V, T, tl)
    up = (g.double() * T).abs()[:, None]
    unrounded = up * (want.abs() / up.clamp(min=1e-30) + q.sum(1, keepdim=True)) * dp[:, None]
    assert ((G - want).abs() <= unrounded + 2.0 ** -8 * want.abs() + 1e-30).all()
    # the products: exact on the G the kernels used
    for got, exact in ((gh, G @ w.double()), (gw, G.T @ h.double())):
        den = exact.norm()
        assert (got.cpu().double() - exact).norm() <= GEMM_FP32_REL_FRO * den + 1e-30
    if bias:
        # FP32 sums of the unrounded G
        tol = unrounded.sum(0) + (N + 8) * 2.0 ** -24 * want.abs().sum(0)
        assert ((gb.cpu().double() - want.sum(0)).abs() <= tol + 1e-30).all()


@pytest.mark.parametrize("T", [1.0, 2.0])
def test_gradient_against_differences(T):
    """Central differences of the 64-bit loss along random directions against the kernel's
    gradients; G's one BF16 rounding (2^-8 at most) bounds what they may differ by."""
    dev = cuda_or_skip()
    h, w, ids, t, b, tl = inputs(40, 48, 260, 9, 6, True)
    ids[3] = -1
    g = torch.randn(40, generator=torch.Generator().manual_seed(7))
    hd, wd, idd, td, bd, gd = on(dev, h, w, ids, t, b, g)
    _, lse = rlk.linear_distill(hd, wd, idd, td, bd, temperature=T)
    grads = rlk.linear_distill_backward(hd, wd, idd, td, lse, gd, bd, temperature=T,
                                        out_dtype=torch.float32)
    G = ref.grad_logits(h, w, ids, t, g, b, T).abs()
    x = [h.double(), w.double(), b.double()]
    for i, grad in enumerate(grads):
        d = torch.randn(x[i].shape, dtype=torch.float64, generator=torch.Generator().manual_seed(8 + i))
        loss = []
        for eps in (1e-5, -1e-5):
            y = list(x)
            y[i] = x[i] + eps * d
            loss.append((g.double() * ref.distill(y[0], y[1], ids, t, y[2], T)[0]).sum())
        slope = (loss[0] - loss[1]) / 2e-5
        d_abs = d.abs()
        if i == 0:
            move = d_abs @ x[1].abs().T
        else:
            move = x[0].abs() @ d_abs.T if i == 1 else d_abs
        tol = 2.0 ** -8 * (G * move).sum() + 1e-6
        assert abs((grad.cpu().double() * d).sum() - slope) <= tol


@pytest.mark.parametrize("N", [1, 31, 100, 300])
def test_one_slot_is_linear_logp(N):
    """K = 1 at T = 1: loss = -logp, the same lse and the same gradients, bit for bit."""
    dev = cuda_or_skip()
    h, w, ids, t, b, _ = on(dev, *inputs(N, 200, 1100, 1, 9, True))
    loss, lse = rlk.linear_distill(h, w, ids, t, b)
    logp, want = rlk.linear_logp(h, w, ids[:, 0], b)
    assert bits_equal(lse, want) and torch.equal(loss, -logp)
    g = torch.randn(N, device=dev)
    gh, gw, _, G = rlk.linear_distill_backward(h, w, ids, t, lse, g, b, return_grad_logits=True)
    wh, ww, _, WG = rlk.linear_logp_backward(h, w, ids[:, 0], lse, -g, b, return_grad_logits=True)
    assert torch.equal(G, WG) and torch.equal(gh, wh) and torch.equal(gw, ww)


def test_rows_do_not_depend_on_the_call():
    """The same rows alone, in chunks over both loops, and in reverse: the same bits."""
    dev = cuda_or_skip()
    h, w, ids, t, b, tl = on(dev, *inputs(400, 136, 1300, 21, 10, True, tail=True, T=1.5))
    ids[::9] = -1
    how = dict(temperature=1.5)
    loss, lse = rlk.linear_distill(h, w, ids, t, b, teacher_lse=tl, **how)
    g = torch.randn(400, device=dev)
    gh = rlk.linear_distill_backward(h, w, ids, t, lse, g, b, teacher_lse=tl, **how)[0]
    for size in (1, 30, 129, 399):
        for r in (0, 57, 400 - size):
            s = slice(r, r + size)
            a, c = rlk.linear_distill(h[s], w, ids[s], t[s], b, teacher_lse=tl[s], **how)
            assert bits_equal(a, loss[s]) and bits_equal(c, lse[s])
            x = rlk.linear_distill_backward(h[s], w, ids[s], t[s], c, g[s], b, teacher_lse=tl[s],
                                            grad_weight=False, **how)[0]
            assert bits_equal(x, gh[s])
    back = torch.arange(399, -1, -1, device=dev)
    a, c = rlk.linear_distill(h[back], w, ids[back], t[back], b, teacher_lse=tl[back], **how)
    assert bits_equal(a[back], loss) and bits_equal(c[back], lse)


def test_layouts_streams_and_repeats():
    """Odd pitches, misaligned operands, strided and expanded lists, leading dims, another
    stream, and repeated calls."""
    dev = cuda_or_skip()
    h, w, ids, t, b, _ = on(dev, *inputs(140, 77, 900, 10, 11, True))
    loss, lse = rlk.linear_distill(h, w, ids, t, b)
    g = torch.randn(140, device=dev)
    want = rlk.linear_distill_backward(h, w, ids, t, lse, g, b)
    wide = torch.zeros(140, 80, dtype=torch.bfloat16, device=dev)
    wide[:, 1:78] = h
    wide_ids = torch.full((140, 15), -1, device=dev)
    wide_ids[:, 2:12] = ids
    wide_t = torch.zeros(140, 13, device=dev)
    wide_t[:, :10] = t
    variants = [(wide[:, 1:78], wide_ids[:, 2:12], wide_t[:, :10]),
                (h.view(7, 20, 77), ids.view(7, 20, 10), t.view(7, 20, 10)),
                (h.t().contiguous().t(), ids.t().contiguous().t(), t)]
    for hv, iv, tv in variants:
        a, c = rlk.linear_distill(hv, w, iv, tv, b)
        assert a.shape == hv.shape[:-1]
        assert bits_equal(a.reshape(-1), loss) and bits_equal(c.reshape(-1), lse)
        x = rlk.linear_distill_backward(hv, w, iv, tv, c, g.view(c.shape), b)
        assert all(bits_equal(p.reshape(q.shape), q) for p, q in zip(x, want))
    one = ids[:1].expand(140, 10)
    a, _ = rlk.linear_distill(h, w, one, t, b)
    assert bits_equal(a, rlk.linear_distill(h, w, one.contiguous(), t, b)[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, c = rlk.linear_distill(h, w, ids, t, b, stream=side)
    side.synchronize()
    assert bits_equal(a, loss) and bits_equal(c, lse)
    for _ in range(5):
        assert bits_equal(rlk.linear_distill(h, w, ids, t, b)[0], loss)
        assert bits_equal(rlk.linear_distill_backward(h, w, ids, t, lse, g, b)[1], want[1])


def test_gradients_asked_for_one_by_one():
    dev = cuda_or_skip()
    h, w, ids, t, b, _ = on(dev, *inputs(70, 64, 400, 6, 12, True))
    _, lse = rlk.linear_distill(h, w, ids, t, b)
    g = torch.randn(70, device=dev)
    every = rlk.linear_distill_backward(h, w, ids, t, lse, g, b)
    for i in range(3):
        want = dict(grad_hidden=i == 0, grad_weight=i == 1, grad_bias=i == 2)
        got = rlk.linear_distill_backward(h, w, ids, t, lse, g, b, **want)
        assert [x is not None for x in got] == [i == j for j in range(3)]
        assert bits_equal(got[i], every[i])


@pytest.mark.parametrize("N,H,V,K,T", [(1, 1, 1, 1, 1.0), (20, 64, 300, 17, 2.0), (130, 72, 1003, 64, 1.0),
                                       (301, 96, 519, 33, 0.5)])
@pytest.mark.parametrize("bias", [False, True])
def test_kept_logits(N, H, V, K, T, bias):
    """The logits the forward keeps are its own, and a backward that reads them gives the bits of
    one that forms them again."""
    dev = cuda_or_skip()
    h, w, ids, t, b, _ = on(dev, *inputs(N, H, V, K, 15, bias, T=T))
    ids[::5] = -1
    ids[1::5, K // 2:] = V
    loss, lse, z = rlk.linear_distill(h, w, ids, t, b, temperature=T, return_logits=True)
    plain = rlk.linear_distill(h, w, ids, t, b, temperature=T)
    assert bits_equal(loss, plain[0]) and bits_equal(lse, plain[1]) and z.shape == (N, V)
    want = h.cpu().double() @ w.cpu().double().T + (b.cpu().double() if bias else 0.0)
    assert ((z.cpu().double() - want).abs().amax(1) <=
            ref.logit_error(h.cpu(), w.cpu(), b.cpu() if bias else None) + 1e-30).all()
    g = torch.randn(N, device=dev)
    for out_dtype in (torch.bfloat16, torch.float32):
        a = rlk.linear_distill_backward(h, w, ids, t, lse, g, b, temperature=T, logits=z,
                                        out_dtype=out_dtype, return_grad_logits=True)
        c = rlk.linear_distill_backward(h, w, ids, t, lse, g, b, temperature=T, out_dtype=out_dtype,
                                        return_grad_logits=True)
        assert all((x is None and y is None) or bits_equal(x, y) for x, y in zip(a, c))
    with pytest.raises(ValueError, match="return_logits"):
        rlk.linear_distill_backward(h, w, ids, t, lse, g, b, logits=z.double())
    got = []
    for keep in (True, False):
        x = [y.clone().requires_grad_() for y in (h, w)]
        loss, _ = rlk.linear_distill_trainable(x[0], x[1], ids, t, b, temperature=T, keep_logits=keep)
        got.append(torch.autograd.grad(loss, x, g))
    assert all(bits_equal(x, y) for x, y in zip(*got))


def test_repeated_calls_of_many_units():
    """Enough units that they are dealt from the counter, and an epilogue whose stores keep the
    memory pipeline full: every call gives the bits of the call that stores no logits."""
    dev = cuda_or_skip()
    N, H, V, K = 2304, 64, 40000, 8
    g = torch.Generator(device=dev).manual_seed(16)
    h = torch.randn(N, H, device=dev, generator=g).bfloat16()
    w = (torch.randn(V, H, device=dev, generator=g) * 0.25).bfloat16()
    ids = torch.randint(V, (N, K), device=dev, generator=g)
    t = torch.randn(N, K, device=dev, generator=g)
    loss, lse = rlk.linear_distill(h, w, ids, t)
    up = torch.randn(N, device=dev, generator=g)
    want = rlk.linear_distill_backward(h, w, ids, t, lse, up)
    for _ in range(40):
        a, b, z = rlk.linear_distill(h, w, ids, t, return_logits=True)
        assert bits_equal(a, loss) and bits_equal(b, lse)
    for kept in (None, z, None, z):
        got = rlk.linear_distill_backward(h, w, ids, t, lse, up, logits=kept)
        assert bits_equal(got[0], want[0]) and bits_equal(got[1], want[1])


def test_trainable():
    """Autograd gives the backward entry's gradients; shared inputs add up; lse is a constant."""
    dev = cuda_or_skip()
    h, w, ids, t, b, tl = on(dev, *inputs(50, 64, 300, 8, 13, True, tail=True, T=2.0))
    for x in (h, w, b):
        x.requires_grad_()
    how = dict(temperature=2.0, teacher_lse=tl)
    loss, lse = rlk.linear_distill_trainable(h.view(5, 10, 64), w, ids.view(5, 10, 8),
                                             t.view(5, 10, 8), b, temperature=2.0,
                                             teacher_lse=tl.view(5, 10))
    assert loss.shape == (5, 10) and not lse.requires_grad
    g = torch.randn(5, 10, device=dev)
    got = torch.autograd.grad(loss, (h, w, b), g)
    d = [x.detach() for x in (h, w, b)]
    want = rlk.linear_distill_backward(d[0], d[1], ids, t, lse.reshape(-1), g.reshape(-1), d[2], **how)
    assert all(bits_equal(x, y.reshape(x.shape)) for x, y in zip(got, want))
    # a broadcast upstream gradient, and only one input that needs a gradient
    loss, lse = rlk.linear_distill_trainable(d[0], w, ids, t, d[2], **how)
    gw, = torch.autograd.grad(loss.sum(), (w,))
    want = rlk.linear_distill_backward(d[0], d[1], ids, t, lse, torch.ones(50, device=dev), d[2], **how)
    assert bits_equal(gw, want[1])
    with pytest.raises(RuntimeError, match="forward-only"):
        rlk.linear_distill(h, w, ids, t, b)


def test_graph_replay():
    dev = cuda_or_skip()
    h, w, ids, t, b, _ = on(dev, *inputs(90, 64, 500, 6, 14, True))
    want, lse = rlk.linear_distill(h, w, ids, t, b)
    g = torch.randn(90, device=dev)
    grads = rlk.linear_distill_backward(h, w, ids, t, lse, g, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, c = rlk.linear_distill(h, w, ids, t, b)
        x = rlk.linear_distill_backward(h, w, ids, t, c, g, b)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert bits_equal(a, want) and bits_equal(c, lse)
        assert all(bits_equal(p, q) for p, q in zip(x, grads))
