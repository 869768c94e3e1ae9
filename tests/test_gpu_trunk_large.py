"""Matrices of more than 2^31 elements: what lies past the 32-bit offsets is found and written."""
import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
from helpers import bits_equal, cuda_or_skip

pytestmark = pytest.mark.gpu


def test_a_table():
    dev = cuda_or_skip()
    V, H = 600_001, 4096                     # 2.46e9 elements
    table = torch.zeros(V, H, dtype=torch.bfloat16, device=dev)
    g = torch.Generator(device=dev).manual_seed(1)
    at = torch.tensor([0, 524_287, 524_288, 524_289, V - 2, V - 1], device=dev)
    table[at] = torch.randn(at.numel(), H, device=dev, generator=g).bfloat16()
    ids = at[torch.tensor([5, 2, 0, 5, 3, 1, 4, 5], device=dev)]
    assert bits_equal(rlk.embedding(ids, table), table[ids])
    del table
    d = torch.randn(ids.numel(), H, device=dev, generator=g).bfloat16()
    grad = rlk.embedding_backward(d, ids, V)
    want = rlk.embedding_backward(d, torch.searchsorted(at, ids), at.numel())
    assert bits_equal(grad[at], want)
    grad[at] = 0
    assert not grad.view(torch.int16).any()
    assert rlk.device_error() == 0


def test_rows_of_a_gated_block():
    dev = cuda_or_skip()
    M, K, F = 70_001, 64, 16_384             # [M, 2, F] is 2.29e9 elements
    g = torch.Generator(device=dev).manual_seed(2)
    x = torch.randn(M, K, device=dev, generator=g).bfloat16()
    w = (torch.randn(2 * F, K, device=dev, generator=g) / 8).bfloat16()
    d = torch.randn(M, F, device=dev, generator=g).bfloat16()
    for keep in ("fp32", "int8", None):
        h = rlk.gated_linear(x, w, keep=keep)
        h, kept = h if keep else (h, None)
        gx, none = rlk.gated_linear_backward(d, x, w, kept=kept, grad_w=False)
        assert none is None
        for a, b in ((0, 50), (65_530, 65_600), (M - 70, M)):
            part = rlk.gated_linear(x[a:b], w, keep=keep)
            part, part_kept = part if keep else (part, None)
            assert bits_equal(part, h[a:b])
            for whole, cut in zip(kept if keep == "int8" else (kept,) if keep else (),
                                  part_kept if keep == "int8" else (part_kept,) if keep else ()):
                assert bits_equal(whole[a:b], cut)
            assert bits_equal(gx[a:b], rlk.gated_linear_backward(d[a:b], x[a:b], w, kept=part_kept, grad_w=False)[0])
        del h, kept, gx
    assert rlk.device_error() == 0


def test_rows_in_8_bits():
    dev = cuda_or_skip()
    M, K = 70_001, 32_768
    x = torch.randn(1000, K, device=dev, generator=torch.Generator(device=dev).manual_seed(3)).bfloat16()
    x = x.repeat(71, 1)[:M]
    q, e = rlk.pack_int8(x)
    want = rlk.pack_int8(x[:1000])
    back = rlk.unpack_int8(q, e)
    del x
    few = rlk.unpack_int8(*want)
    for a in (0, 65_000, 69_000):
        assert torch.equal(q[a:a + 1000], want[0]) and torch.equal(e[a:a + 1000], want[1])
        assert bits_equal(back[a:a + 1000], few)
    assert bits_equal(back[-1], few[0]) and rlk.device_error() == 0
