"""The trunk's operators as they are used: together, on streams of their own, in graphs, from several
threads, between guard bands."""
import importlib.util
import os
import threading

import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
import trunk_reference as ref
from helpers import bits_equal, cuda_or_skip
from test_gpu_sample_distill_guard_bands import Guarded

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
LONG = 40_000_000        # cycles, some 20 ms


def load_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "tied_policy_training.py")
    spec = importlib.util.spec_from_file_location("tied_policy_training", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


# ------------------------------------------------------------------ together
def exact_gradients(tokens, targets, master):
    """The same network in 64 bits, by autograd, from the bf16 weights."""
    table, w_in, w_out = (m.bfloat16().double().requires_grad_() for m in master)
    x = table[tokens]
    z = x @ w_in.t()
    f = w_in.size(0) // 2
    h = torch.nn.functional.silu(z[..., :f]) * z[..., f:]
    logits = (x + h @ w_out.t()) @ table.t()
    loss = -torch.log_softmax(logits, -1).gather(-1, targets[..., None]).mean()
    return loss.detach(), torch.autograd.grad(loss, (table, w_in, w_out))


@pytest.mark.parametrize("checkpoint", [None, "fp32", "again", "int8"])
@pytest.mark.parametrize("batch,length,sizes", [(1, 1, dict(hidden=64, inner=96, vocab=300)),
                                                (3, 37, dict(hidden=100, inner=130, vocab=1001)),
                                                (4, 128, dict(hidden=256, inner=700, vocab=5000))])
def test_a_training_step_of_them_all(batch, length, sizes, checkpoint):
    cuda_or_skip()
    example = load_example()
    master = example.start(**sizes)
    g = torch.Generator(device="cuda").manual_seed(7)
    vocab = sizes["vocab"]
    tokens = torch.randint(vocab, (batch, length), device="cuda", generator=g)
    tokens[:, length // 3:length // 2] = 5                       # one token many times
    targets = torch.randint(vocab, (batch, length), device="cuda", generator=g)
    loss, grads = example.gradients(tokens, targets, master, checkpoint)
    again = example.gradients(tokens, targets, master, checkpoint)
    assert bits_equal(loss, again[0]) and all(bits_equal(a, b) for a, b in zip(grads, again[1]))
    exact_loss, exact = exact_gradients(tokens, targets, master)
    # x, h, y, x + y and on the way back dlogits, d(x + y), dh, dz, dx and the gradient itself are
    # rounded to BF16: ten times at most 2^-8 relative, doubled for the maps between.  The tied
    # table's two gradients are added in BF16 (one more).  8 bits: x twice, g, u and h off by at
    # most half a step, 2^-7 of a block's largest, taken as three root mean squares.
    bound = 11 * 2 * 2.0 ** -8 + (5 * 3 * 2.0 ** -7 if checkpoint == "int8" else 0)
    assert abs(loss.item() - exact_loss.item()) <= 0.01 * abs(exact_loss.item())
    for a, b in zip(grads, exact):
        assert (a.double() - b).norm() <= bound * b.norm()
    if checkpoint == "again":
        kept = example.gradients(tokens, targets, master, "fp32")
        assert bits_equal(loss, kept[0]) and all(bits_equal(a, b) for a, b in zip(grads, kept[1]))


def test_the_example_runs_and_repeats():
    cuda_or_skip()
    example = load_example()
    for checkpoint in (None, "int8"):
        losses, master = example.train(steps=3, batch=2, length=40, checkpoint=checkpoint, hidden=96, inner=100,
                                       vocab=1000)
        again = example.train(steps=3, batch=2, length=40, checkpoint=checkpoint, hidden=96, inner=100, vocab=1000)
        assert losses == again[0] and all(bits_equal(a, b) for a, b in zip(master, again[1]))


def test_accumulated_table_gradients():
    """Micro-batches of a tied table: both of its gradients added to one FP32 tensor."""
    dev = cuda_or_skip()
    g = torch.Generator(device=dev).manual_seed(8)
    V, H = 900, 64
    table = torch.randn(V, H, device=dev, generator=g).bfloat16()
    total = torch.zeros(V, H, device=dev)
    want = torch.zeros(V, H, device=dev, dtype=torch.float64)
    for n in (50, 1, 200):
        ids = torch.randint(V, (n,), device=dev, generator=g)
        x = rlk.embedding(ids, table, 2.0)
        target = torch.randint(V, (n,), device=dev, generator=g)
        _, lse = rlk.linear_logp(x, table, target)
        up = torch.randn(n, device=dev, generator=g)
        gx, gw, _ = rlk.linear_logp_backward(x, table, target, lse, up, out_dtype=FP32)
        total += gw
        rlk.embedding_grad_accum_fp32_(total, gx, ids, 2.0)
        want += gw.double() + ref.embedding_grad(ids, gx, V, 2.0)
    # FP32 sums of at most 200 + 6 terms
    assert (total.double() - want).norm() <= 256 * 2.0 ** -24 * want.norm()


# ------------------------------------------------------------------ streams, graphs, threads
def entries(dev):
    """name -> (call of a stream and its inputs, inputs); strided operands, so every call copies some."""
    g = torch.Generator(device=dev).manual_seed(0)

    def numbers(*shape, dtype=BF16):
        return torch.randn(*shape, device=dev, generator=g).to(dtype).t().contiguous().t()

    x, w, d = numbers(150, 72), numbers(180, 72), numbers(150, 90)
    ids = torch.randint(300, (150, 2), device=dev, generator=g)[:, 1]
    table, rows = numbers(300, 40), numbers(150, 40)
    total = torch.randn(300, 40, device=dev, generator=g)
    kept32 = rlk.gated_linear(x, w, keep="fp32")[1]
    kept8 = rlk.gated_linear(x, w, keep="int8")[1]
    q, e = rlk.pack_int8(numbers(150, 70))
    return {
        "embedding": (lambda s, *a: rlk.embedding(*a, 2.0, stream=s), (ids, table)),
        "embedding_backward": (lambda s, *a: rlk.embedding_backward(*a, 300, 2.0, stream=s), (rows, ids)),
        "embedding_accum": (lambda s, t, *a: rlk.embedding_grad_accum_fp32_(t, *a, stream=s), (total, rows, ids)),
        "pack_int8": (lambda s, x: rlk.pack_int8(x, stream=s), (x,)),
        "unpack_int8": (lambda s, *a: rlk.unpack_int8(*a, stream=s), (q, e)),
        "gated_linear": (lambda s, *a: rlk.gated_linear(*a, stream=s), (x, w)),
        "gated_linear fp32": (lambda s, *a: rlk.gated_linear(*a, keep="fp32", stream=s), (x, w)),
        "gated_linear int8": (lambda s, *a: flat(rlk.gated_linear(*a, keep="int8", stream=s)), (x, w)),
        "backward again": (lambda s, *a: rlk.gated_linear_backward(*a, stream=s), (d, x, w)),
        "backward fp32": (lambda s, d, x, w, k: rlk.gated_linear_backward(d, x, w, kept=k, stream=s), (d, x, w, kept32)),
        "backward int8": (lambda s, d, x, w, q, e: rlk.gated_linear_backward(d, x, w, kept=(q, e), stream=s),
                          (d, x, w, *kept8)),
    }


def flat(out):
    return [t for o in (out if isinstance(out, (tuple, list)) else (out,))
            for t in (flat(o) if isinstance(o, (tuple, list)) else (o,))]


NAMES = ["embedding", "embedding_backward", "embedding_accum", "pack_int8", "unpack_int8", "gated_linear",
         "gated_linear fp32", "gated_linear int8", "backward again", "backward fp32", "backward int8"]


def same_layout(t):
    return torch.empty_strided(t.size(), t.stride(), dtype=t.dtype, device=t.device).copy_(t)


def fill(dev):
    for _ in range(3):                        # takes over whatever memory was given back
        held = [torch.full((n,), 0x7f, dtype=torch.uint8, device=dev) for n in [512 << i for i in range(16)] * 4]
        del held


@pytest.mark.parametrize("name", NAMES)
def test_a_call_on_another_stream(name):
    dev = cuda_or_skip()
    of = entries(dev)
    assert list(of) == NAMES
    call, inputs = of[name]
    want = [t.clone() for t in flat(call(None, *(same_layout(t) for t in inputs)))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for late in (False, True):
        mine = [same_layout(t) for t in inputs]
        side.wait_stream(torch.cuda.current_stream())
        if late:
            torch.cuda._sleep(LONG)           # the current stream is behind: nothing may be left to it
        else:
            with torch.cuda.stream(side):     # the other stream is: nothing of its may be taken
                torch.cuda._sleep(LONG)
        got = flat(call(side, *mine))
        del mine
        fill(dev)
        if late:
            side.synchronize()
        else:
            torch.cuda.current_stream().wait_stream(side)
        assert all(bits_equal(a, b) for a, b in zip(got, want))
        copies = [torch.empty_like(b) for b in want]
        torch.cuda._sleep(LONG)               # outputs that the current stream reads late may be dropped
        for c, a in zip(copies, got):
            c.copy_(a)
        del got, a
        with torch.cuda.stream(side):
            fill(dev)
        torch.cuda.synchronize()
        assert all(bits_equal(a, b) for a, b in zip(copies, want))
    assert rlk.device_error() == 0


@pytest.mark.parametrize("M,K,F", [(1, 64, 128), (100, 200, 130), (300, 256, 1000), (2600, 64, 7100)])
def test_captured_and_replayed(M, K, F):
    """Two graphs of a whole step, replayed in turn with new inputs in their buffers (the largest: tiles
    handed out from the workspace's counter)."""
    dev = cuda_or_skip()
    V = 700

    def inputs(seed):
        g = torch.Generator(device=dev).manual_seed(seed)
        return [torch.randint(V, (M,), device=dev, generator=g),
                torch.randn(V, K, device=dev, generator=g).bfloat16(),
                (torch.randn(2 * F, K, device=dev, generator=g) / K ** 0.5).bfloat16(),
                torch.randn(M, F, device=dev, generator=g).bfloat16()]

    def step(ids, table, w, d):
        x = rlk.embedding(ids, table, 1.5)
        h, kept32 = rlk.gated_linear(x, w, keep="fp32")
        _, kept8 = rlk.gated_linear(x, w, keep="int8")
        held = rlk.unpack_int8(*rlk.pack_int8(x))
        out = [h]
        for kept, at in ((None, x), (kept32, x), (kept8, held)):
            gx, gw = rlk.gated_linear_backward(d, at, w, kept=kept)
            out += [gx, gw, rlk.embedding_backward(gx, ids, V, 1.5)]
        return out

    a, b = inputs(1), inputs(2)
    want = [[t.clone() for t in step(*i)] for i in (a, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*a)
    torch.cuda.current_stream().wait_stream(side)
    graphs, buffers = [], []
    for _ in range(2):
        own = [t.clone() for t in a]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step(*own)
        graphs.append((graph, outs))
        buffers.append(own)
    for turn in range(4):
        which = turn % 2
        for t, new in zip(buffers[which], (a, b)[turn // 2 ^ which]):
            t.copy_(new)
        graphs[which][0].replay()
        if turn % 2 == 0:
            continue
        torch.cuda.synchronize()
        for k in range(2):
            for got, exp in zip(graphs[k][1], want[turn // 2 ^ k]):
                assert bits_equal(got, exp)
    assert rlk.device_error() == 0


@pytest.mark.parametrize("checkpoint", ["fp32", "int8", "again"])
@pytest.mark.parametrize("n,K,F", [(1, 64, 96), (100, 72, 130), (300, 256, 500)])
def test_captured_through_autograd(n, K, F, checkpoint):
    """Forward and backward through autograd in one graph, replayed with new numbers in its buffers.
    The graph has leaves of its own: a leaf that an eager graph still holds keeps that graph's stream."""
    dev = cuda_or_skip()
    V = 500

    def inputs(seed):
        g = torch.Generator(device=dev).manual_seed(seed)
        return [torch.randint(-1, V, (n,), device=dev, generator=g),
                torch.randn(V, K, device=dev, generator=g).bfloat16(),
                (torch.randn(2 * F, K, device=dev, generator=g) / K ** 0.5).bfloat16(),
                (torch.randn(K, F, device=dev, generator=g) / F ** 0.5).bfloat16(),
                torch.randn(n, K, device=dev, generator=g).bfloat16()]

    def step(ids, table, w_in, w_out, up):
        leaves = [t.requires_grad_() for t in (table, w_in, w_out)]
        x = rlk.embedding_trainable(ids, table, 1.5)
        h = rlk.gated_linear_trainable(x, w_in, checkpoint=checkpoint)
        y = rlk.det_linear_trainable(h, w_out, checkpoint="int8" if checkpoint == "int8" else None)
        return [y.detach(), *torch.autograd.grad(y, leaves, up)]

    a, b = inputs(5), inputs(6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [[t.clone() for t in step(*(t.clone() for t in i))] for i in (a, b)]
    torch.cuda.current_stream().wait_stream(side)
    own = [t.clone() for t in a]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*own)
    for i, exp in ((b, want[1]), (a, want[0]), (b, want[1])):
        with torch.no_grad():
            for t, new in zip(own, i):
                t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, exp):
            assert bits_equal(x, y)
    assert rlk.device_error() == 0


def test_threads_on_their_own_streams():
    dev = cuda_or_skip()
    of = entries(dev)
    want = {n: [t.clone() for t in flat(call(None, *(same_layout(i) for i in inputs)))]
            for n, (call, inputs) in of.items()}
    torch.cuda.synchronize()
    errors = []

    def worker(k):
        try:
            stream = torch.cuda.Stream(device=dev)
            with torch.cuda.stream(stream):
                for turn in range(3):
                    names = NAMES[k:] + NAMES[:k]
                    for n in names:
                        call, inputs = of[n]
                        got = flat(call(None, *(same_layout(i) for i in inputs)))
                        stream.synchronize()
                        if not all(bits_equal(a, b) for a, b in zip(got, want[n])):
                            errors.append((n, turn))
        except Exception as e:               # noqa: BLE001 (shown in the test's own thread)
            errors.append(e)

    threads = [threading.Thread(target=worker, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    assert rlk.device_error() == 0


@pytest.mark.parametrize("name", ["embedding", "gated_linear", "gated_linear int8"])
def test_second_derivative_is_refused(name):
    dev = cuda_or_skip()
    w = torch.randn(300, 32, device=dev).bfloat16().requires_grad_()
    x = torch.randn(20, 32, device=dev).bfloat16()
    out = rlk.embedding_trainable(torch.arange(20, device=dev), w) if name == "embedding" else \
        rlk.gated_linear_trainable(x, w, checkpoint="int8" if "int8" in name else None)
    up = torch.ones_like(out).requires_grad_()
    grad, = torch.autograd.grad(out, (w,), up, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grad.float().square().sum().backward()


# ------------------------------------------------------------------ cliffs
def median_us(call, reps=11):
    times = []
    for _ in range(3):
        call()
    for _ in range(reps):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda._sleep(100_000)            # the host's launches are not what is timed
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    return sorted(times)[reps // 2]


def test_odd_widths_stay_off_the_cliff():
    """Ratios of times in one process: an odd width costs at most half as much again as an even one
    (it took two to five times as much with single elements from each row's thread)."""
    dev = cuda_or_skip()
    g = torch.Generator(device=dev).manual_seed(9)
    times = {}
    for F in (5464, 5461):
        x = torch.randn(2000, 2048, device=dev, generator=g).bfloat16()
        w = torch.randn(2 * F, 2048, device=dev, generator=g).bfloat16()
        d = torch.randn(2000, F, device=dev, generator=g).bfloat16()
        times[F] = [median_us(lambda: rlk.gated_linear(x, w)), median_us(lambda: rlk.gated_linear_backward(d, x, w)),
                    median_us(lambda: rlk.det_gemm_db(x[:255], d[:255])), median_us(lambda: rlk.det_linear(x, w[:F]))]
    assert all(b <= 1.5 * a for a, b in zip(times[5464], times[5461])), times


# ------------------------------------------------------------------ guard bands, through the C ABI
def ptr(t):
    return None if t is None else t.data_ptr()


def pitched(b, rows, cols, pitch, dtype):
    """A guarded [rows, cols] output of a wider pitch, and the view of its padding."""
    raw = b.take(rows * pitch * dtype.itemsize, dtype, (rows, pitch))
    return raw[:, :cols], raw[:, cols:]


def untouched(*pads):
    return all((p.contiguous().view(torch.uint8) == 0xA5).all() for p in pads)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (FP32, FP32), (BF16, FP32), (FP32, BF16)])
@pytest.mark.parametrize("n,V,H", [(1, 1, 1), (70, 3, 33), (300, 1030, 64), (5, 2050, 2056)])
def test_embedding_guard_bands(n, V, H, dtype, out_dtype, wide):
    dev = cuda_or_skip()
    g = torch.Generator(device=dev).manual_seed(H)
    ids = torch.randint(-1, V + 1, (n,), device=dev, generator=g)
    ids[: n // 2] = 0
    w = torch.randn(V, H, device=dev, generator=g).to(dtype)
    d = torch.randn(n, H, device=dev, generator=g).to(dtype)
    b, lib, stream = Guarded(dev), rlk.lib(), rlk._stream_ptr(None)
    pitch = H + (8 if wide else 0)
    out, pad = pitched(b, n, H, pitch, out_dtype)
    assert lib.rlk_embedding(ptr(ids), 1, n, ptr(w), rlk._DT[dtype], V, H, H, 0.5, ptr(out), rlk._DT[out_dtype], pitch,
                             stream) == 0
    size = lib.rlk_embedding_backward_workspace_size(n, V, H)
    ws = b.take(size)
    table, tpad = pitched(b, V, H, pitch, out_dtype)
    args = (ptr(ids), 1, n, ptr(d), rlk._DT[dtype], H, H, 0.5)
    assert lib.rlk_embedding_backward(*args, ptr(table), rlk._DT[out_dtype], V, pitch, 0, ptr(ws), size, stream) == 0
    b.check()
    assert bits_equal(out.contiguous(), rlk.embedding(ids, w, 0.5, out_dtype=out_dtype))
    want = rlk.embedding_backward(d, ids, V, 0.5, out_dtype)
    assert bits_equal(table.contiguous(), want) and untouched(pad, tpad)
    if out_dtype == FP32:
        before = torch.randn(V, H, device=dev, generator=g)
        table.copy_(before)
        assert lib.rlk_embedding_backward(*args, ptr(table), rlk.RLK_FP32, V, pitch, 1, ptr(ws), size, stream) == 0
        b.check()
        assert bits_equal(table.contiguous(), rlk.embedding_grad_accum_fp32_(before, d, ids, 0.5)) and untouched(tpad)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("rows,cols,extra", [(1, 1, 0), (3, 33, 16), (130, 128, 0), (65, 2081, 32), (7, 4096, 16)])
def test_int8_guard_bands(rows, cols, extra, dtype):
    dev = cuda_or_skip()
    x = torch.randn(rows, cols, device=dev, generator=torch.Generator(device=dev).manual_seed(cols)).to(dtype)
    blocks = -(-cols // 32)
    b, lib, stream = Guarded(dev), rlk.lib(), rlk._stream_ptr(None)
    q, qpad = pitched(b, rows, 32 * blocks, 32 * blocks + extra, torch.int8)
    e, epad = pitched(b, rows, blocks, blocks + extra // 16, torch.uint8)
    pitch = cols + extra
    back, bpad = pitched(b, rows, cols, pitch, dtype)
    assert lib.rlk_pack_int8(ptr(x), rlk._DT[dtype], rows, cols, cols, ptr(q), q.stride(0), ptr(e), e.stride(0),
                             stream) == 0
    assert lib.rlk_unpack_int8(ptr(q), rows, cols, q.stride(0), ptr(e), e.stride(0), ptr(back), rlk._DT[dtype], pitch,
                               stream) == 0
    b.check()
    want = rlk.pack_int8(x)
    assert torch.equal(q[:, :cols], want[0]) and torch.equal(e, want[1]) and not q[:, cols:].any()
    assert bits_equal(back.contiguous(), rlk.unpack_int8(*want, dtype)) and untouched(qpad, epad, bpad)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("M,K,F", [(1, 1, 1), (33, 40, 33), (128, 72, 130), (129, 33, 1), (260, 64, 100), (300, 136, 257)])
def test_gated_guard_bands(M, K, F, dtype, wide):
    dev = cuda_or_skip()
    g = torch.Generator(device=dev).manual_seed(F)
    x = torch.randn(M, K, device=dev, generator=g).bfloat16()
    w = torch.randn(2 * F, K, device=dev, generator=g).bfloat16()
    d = torch.randn(M, F, device=dev, generator=g).to(dtype)
    Fp, lib, stream = -(-F // 32) * 32, rlk.lib(), rlk._stream_ptr(None)
    extra = 8 if wide else 0
    dt = rlk._DT[dtype]
    for keep in (0, 1, 2):
        b = Guarded(dev)
        size = lib.rlk_gated_linear_workspace_size(ptr(x), M, K, K, ptr(w), F, K)
        ws = b.take(size)
        h, hpad = pitched(b, M, F, F + extra, dtype)
        kept = b.take(M * 2 * Fp * (4 if keep == 1 else 1), FP32 if keep == 1 else torch.int8, (M, 2, Fp)) if keep else None
        e = b.take(M * Fp // 16, torch.uint8, (M, 2, Fp // 32)) if keep == 2 else None
        assert lib.rlk_gated_linear(ptr(x), M, K, K, ptr(w), F, K, 0, ptr(h), dt, F + extra, keep, ptr(kept), ptr(e),
                                    ptr(ws), size, stream) == 0
        size = lib.rlk_gated_linear_backward_workspace_size(ptr(x), M, K, K, ptr(w), F, K)
        ws = b.take(size)
        dx, xpad = pitched(b, M, K, K + extra, dtype)
        dw, wpad = pitched(b, 2 * F, K, K + extra, dtype)
        assert lib.rlk_gated_linear_backward(ptr(d), dt, M, F, F, ptr(x), K, K, ptr(w), K, 0, keep, ptr(kept), ptr(e),
                                             ptr(dx), dt, K + extra, ptr(dw), dt, K + extra, ptr(ws), size, stream) == 0
        b.check()
        what = (None, "fp32", "int8")[keep]
        want = rlk.gated_linear(x, w, out_dtype=dtype, keep=what)
        want, parts = want if keep else (want, None)
        assert bits_equal(h.contiguous(), want)
        for got, exp in zip((kept, e), flat(parts) if keep else ()):
            assert bits_equal(got + 0, exp + 0)
        grads = rlk.gated_linear_backward(d, x, w, kept=parts, out_dtype=dtype)
        assert bits_equal(dx.contiguous(), grads[0]) and bits_equal(dw.contiguous(), grads[1])
        assert untouched(hpad, xpad, wpad)


def test_operands_that_a_product_does_not_read_may_be_missing():
    dev = cuda_or_skip()
    g = torch.Generator(device=dev).manual_seed(3)
    M, K, F = 40, 64, 96
    x = torch.randn(M, K, device=dev, generator=g).bfloat16()
    w = torch.randn(2 * F, K, device=dev, generator=g).bfloat16()
    d = torch.randn(M, F, device=dev, generator=g).bfloat16()
    kept = rlk.gated_linear(x, w, keep="int8")[1]
    want = rlk.gated_linear_backward(d, x, w, kept=kept)
    lib, stream = rlk.lib(), rlk._stream_ptr(None)
    for with_x in (False, True):
        b = Guarded(dev)
        px, pw = (x.data_ptr(), None) if with_x else (None, w.data_ptr())
        size = lib.rlk_gated_linear_backward_workspace_size(px, M, K, K, pw, F, K)
        ws = b.take(size)
        out = b.take(2 * (2 * F if with_x else M) * K, BF16, (2 * F if with_x else M, K))
        dx, dw = (None, out.data_ptr()) if with_x else (out.data_ptr(), None)
        assert lib.rlk_gated_linear_backward(ptr(d), 0, M, F, F, px, K, K, pw, K, 0, 2, ptr(kept[0]), ptr(kept[1]), dx, 0, K,
                                             dw, 0, K, ptr(ws), size, stream) == 0
        b.check()
        assert bits_equal(out, want[1 if with_x else 0])


def test_operands_on_one_device_only():
    dev = cuda_or_skip()
    x = torch.randn(4, 8, device=dev).bfloat16()
    for call in (lambda: rlk.gated_linear(x, x.cpu()), lambda: rlk.embedding(torch.zeros(2, dtype=torch.int64), x),
                 lambda: rlk.embedding_backward(x, torch.zeros(4, dtype=torch.int64), 5),
                 lambda: rlk.unpack_int8(x.to(torch.int8), torch.zeros(4, 1, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call()
