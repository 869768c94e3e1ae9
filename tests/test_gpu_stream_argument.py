"""stream=: what a call makes and drops is neither read unfinished nor reused early, whatever the
current stream does meanwhile, and inputs and outputs may be dropped on either side."""
import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
from helpers import bits_equal, cuda_or_skip

pytestmark = pytest.mark.gpu
LONG = 40_000_000        # cycles, some 20 ms


def entries(dev):
    """name -> (call of a stream and its inputs, inputs): strided operands, so every call copies some."""
    g = torch.Generator(device=dev).manual_seed(0)

    def bf16(*shape):
        return torch.randn(*shape, device=dev, generator=g).bfloat16().t().contiguous().t()

    h, w, x = bf16(150, 72), bf16(3001, 72), bf16(72, 90)
    up = torch.randn(150, 2, device=dev, generator=g)[:, 0]
    target = torch.randint(3001, (150,), device=dev, generator=g)
    ids = torch.randint(3001, (7, 150), device=dev, generator=g).t()
    t = torch.randn(7, 150, device=dev, generator=g).t()
    lse = rlk.linear_logp(h, w, target)[1]
    dlse = rlk.linear_distill(h, w, ids, t)[1]
    z = torch.randn(20011, 120, device=dev, generator=g).t()
    u = torch.rand(120, 2, device=dev, generator=g, dtype=torch.float64)[:, 1]
    tau = torch.rand(120, 2, device=dev, generator=g)[:, 1] + 0.5
    c = torch.randn(150, 90, device=dev, generator=g)
    dc, dy = bf16(150, 90), bf16(150, 3001)
    parts = torch.randn(90, 3, 150, device=dev, generator=g).permute(1, 2, 0)
    j0, j1, v0, v1 = rlk.vocab_shard_range(3001, 2, 0)
    k0, k1, _, v2 = rlk.vocab_shard_range(3001, 2, 1)
    shard = w[v0:v1].t().contiguous().t()
    both = [rlk.linear_logp_shard_partials(h, s, target, 3001, a, b, ld_partials=max(j1 - j0, k1 - k0))
            for s, a, b in ((w[v0:v1], j0, j1), (w[v1:v2], k0, k1))]
    gp, gz = (torch.stack([b[i] for b in both]) for i in range(2))
    return {
        "linear_logp": (lambda s, h, w, y: rlk.linear_logp(h, w, y, stream=s), (h, w, target)),
        "shard_partials": (lambda s, h, w, y: rlk.linear_logp_shard_partials(
            h, w, y, 3001, j0, j1, stream=s), (h, shard, target)),
        "combine_shards": (lambda s, p, z, y: rlk.linear_logp_combine_shards(
            p, z, [j0, j1, k1], y, 3001, stream=s), (gp, gz, target)),
        "linear_logp_backward": (lambda s, h, w, y, l, g: rlk.linear_logp_backward(
            h, w, y, l, g, stream=s)[:2], (h, w, target, lse, up)),
        "sample short": (lambda s, z, u, tau: rlk.sample_logits(
            z, u, temperature=tau, top_k=30, stream=s), (z[:20], u[:20], tau[:20])),
        "sample streaming": (lambda s, z, u, tau: rlk.sample_logits(
            z, u, temperature=tau, top_p=0.9, stream=s), (z, u, tau)),
        "linear_distill": (lambda s, *a: rlk.linear_distill(*a, stream=s), (h, w, ids, t)),
        "linear_distill kept": (lambda s, *a: rlk.linear_distill(*a, return_logits=True, stream=s),
                                (h, w, ids, t)),
        "linear_distill_backward": (lambda s, *a: rlk.linear_distill_backward(*a, stream=s)[:2],
                                    (h, w, ids, t, dlse, up)),
        "det_gemm_fwd": (lambda s, *a: rlk.det_gemm_fwd(*a, stream=s), (h, x)),
        "det_gemm_da": (lambda s, *a: rlk.det_gemm_da(*a, stream=s), (dc, x)),
        "det_gemm_db": (lambda s, *a: rlk.det_gemm_db(*a, stream=s), (h, dc)),
        "det_gemm_accum": (lambda s, c, *a: rlk.det_gemm_fwd_accum_fp32_(c, *a, stream=s), (c, h, x)),
        "det_gemm_backward": (lambda s, *a: rlk.det_gemm_backward(*a, stream=s), (dc, h, x)),
        "det_linear": (lambda s, *a: rlk.det_linear(*a, stream=s), (h, w)),
        "det_linear_dx": (lambda s, *a: rlk.det_linear_dx(*a, stream=s), (dy, w)),
        "det_linear_dw": (lambda s, *a: rlk.det_linear_dw(*a, stream=s), (dy, h)),
        "det_linear_backward": (lambda s, *a: rlk.det_linear_backward(*a, stream=s), (dy, h, w)),
        "sum_partials": (lambda s, p: rlk.sum_partials_ordered(p, stream=s), (parts,)),
    }


NAMES = ["linear_logp", "shard_partials", "combine_shards", "linear_logp_backward", "sample short",
         "sample streaming", "linear_distill", "linear_distill kept", "linear_distill_backward",
         "det_gemm_fwd", "det_gemm_da", "det_gemm_db", "det_gemm_accum", "det_gemm_backward",
         "det_linear", "det_linear_dx", "det_linear_dw", "det_linear_backward", "sum_partials"]


def outputs(out):
    return list(out) if isinstance(out, tuple) else [out]


def same_layout(t):
    return torch.empty_strided(t.size(), t.stride(), dtype=t.dtype, device=t.device).copy_(t)


@pytest.mark.parametrize("name", NAMES)
def test_the_current_stream_goes_on(name):
    dev = cuda_or_skip()
    of = entries(dev)
    assert list(of) == NAMES
    call, inputs = of[name]
    want = [x.clone() for x in outputs(call(None, *(same_layout(x) for x in inputs)))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for late in (False, True):
        mine = [same_layout(x) for x in inputs]
        side.wait_stream(torch.cuda.current_stream())
        if late:
            torch.cuda._sleep(LONG)           # the current stream is behind: nothing may be left to it
        else:
            with torch.cuda.stream(side):     # the other stream is: nothing of its may be taken
                torch.cuda._sleep(LONG)
        got = outputs(call(side, *mine))
        del mine
        for _ in range(3):                    # takes over whatever memory was given back
            fill = [torch.full((n,), 0x7f, dtype=torch.uint8, device=dev)
                    for n in [512 << i for i in range(16)] * 4]
            del fill
        if late:
            side.synchronize()
        else:
            torch.cuda.current_stream().wait_stream(side)
        assert all(bits_equal(a, b) for a, b in zip(got, want))
        # outputs that the current stream reads late may be dropped at once
        copies = [torch.empty_like(b) for b in want]
        torch.cuda._sleep(LONG)
        for c, a in zip(copies, got):
            c.copy_(a)
        del got, a
        with torch.cuda.stream(side):
            for _ in range(3):
                fill = [torch.full((n,), 0x7f, dtype=torch.uint8, device=dev)
                        for n in [512 << i for i in range(16)] * 4]
                del fill
        torch.cuda.synchronize()
        assert all(bits_equal(a, b) for a, b in zip(copies, want))
    assert rlk.device_error() == 0


def test_a_prepared_call_may_be_dropped():
    dev = cuda_or_skip()
    g = torch.Generator(device=dev).manual_seed(1)
    h = torch.randn(300, 64, device=dev, generator=g).bfloat16()
    w = torch.randn(3001, 64, device=dev, generator=g).bfloat16()
    y = torch.randint(3001, (300,), device=dev, generator=g)
    want = [x.clone() for x in rlk.LinearLogpCall(h, w, y)()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG)
    got = rlk.LinearLogpCall(h.clone(), w.clone(), y.clone())(stream=side)
    fill = [torch.full((n,), 0x7f, dtype=torch.uint8, device=dev) for n in [512 << i for i in range(16)] * 4]
    del fill
    torch.cuda.synchronize()
    assert all(bits_equal(a, b) for a, b in zip(got, want))
