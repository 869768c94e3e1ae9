"""Embedding lookup and gradient against their definitions."""
import math

import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
import trunk_reference as ref
from helpers import bits_equal, cuda_or_skip

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


def some_ids(n, V, seed=0, common=0.3):
    """Ids of which a share is one id and some name no row."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(V, (n,), generator=g)
    r = torch.rand(n, generator=g)
    ids[r < common] = V // 2
    ids[r > 0.95] = torch.tensor([-1, V, -(1 << 40), 1 << 40])[torch.randint(4, (n,), generator=g)][r > 0.95]
    return ids.to(cuda_or_skip())


def numbers(*shape, dtype=BF16, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).to(cuda_or_skip())


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, None), (FP32, None), (BF16, FP32), (FP32, BF16)])
@pytest.mark.parametrize("n,V,H", [(1, 1, 1), (3, 5, 7), (65, 100, 64), (2, 300, 1000), (257, 1025, 129),
                                   (40, 77, 2056), (9, 11, 5001)])
@pytest.mark.parametrize("scale", [1.0, -0.3, math.sqrt(1000)])
def test_lookup(n, V, H, scale, dtype, out_dtype):
    ids, w = some_ids(n, V), numbers(V, H, dtype=dtype)
    out = rlk.embedding(ids, w, scale, out_dtype=out_dtype)
    known = (ids >= 0) & (ids < V)
    want = w[torch.where(known, ids, 0)].float() * scale              # one product, one rounding
    want = torch.where(known[:, None], want, 0.0).to(out_dtype or dtype)
    assert bits_equal(out, want)
    assert rlk.device_error() == 0


def test_lookup_of_any_layout():
    w = numbers(50, 96)
    ids = some_ids(24, 50)
    want = rlk.embedding(ids, w)
    wide = numbers(50, 131)
    wide[:, 1:97] = w
    assert bits_equal(rlk.embedding(ids, wide[:, 1:97]), want)           # odd pitch, odd start
    assert bits_equal(rlk.embedding(ids, w.t().contiguous().t()), want)  # column-major: copied
    assert bits_equal(rlk.embedding(ids.view(2, 3, 4), w), want.view(2, 3, 4, 96))
    assert bits_equal(rlk.embedding(torch.stack([ids, ids], 1)[:, 0], w), want)          # strided
    assert bits_equal(rlk.embedding(ids[3].expand(7), w), want[3].expand(7, 96))         # stride 0
    assert bits_equal(rlk.embedding(ids[3], w), want[3])
    assert rlk.embedding(ids[:0], w).shape == (0, 96)


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (FP32, FP32), (BF16, FP32), (FP32, BF16)])
@pytest.mark.parametrize("n,V,H", [(1, 1, 1), (3, 5, 7), (64, 3, 40), (65, 1, 33), (200, 1024, 64),
                                   (300, 1025, 129), (1500, 2500, 100), (700, 3, 1030)])
def test_gradient_has_the_defined_order(n, V, H, dtype, out_dtype):
    ids, d = some_ids(n, V, 2), numbers(n, H, dtype=dtype, seed=3)
    out = rlk.embedding_backward(d, ids, V, 0.7, out_dtype)
    want = ref.embedding_grad_fp32(ids, d, V, 0.7).to(out_dtype).to(out.device)
    assert bits_equal(out + 0.0, want + 0.0)          # (a sum of -0 alone is 0 in one and -0 in neither)
    assert rlk.device_error() == 0


@pytest.mark.parametrize("out_dtype", [BF16, FP32])
@pytest.mark.parametrize("n,V,H,common", [(5000, 3000, 64, 0.9), (40000, 700, 24, 0.5), (100000, 50000, 8, 0.2),
                                          (33000, 1, 9, 0.0), (20000, 100001, 16, 0.01)])
def test_gradient_of_many_rows(n, V, H, common, out_dtype):
    ids, d = some_ids(n, V, 4, common), numbers(n, H, dtype=FP32, seed=5)
    out = rlk.embedding_backward(d, ids, V, 1.5, out_dtype).double()
    want = ref.embedding_grad(ids, d, V, 1.5)
    # an FP32 sum of c numbers in groups: at most 64 + c / 64 additions deep, half a step of
    # 2^-24 of the running sum (at most the sum of magnitudes) each; then scale and the output
    size = ref.embedding_grad(ids, d.abs(), V, 1.5)
    count = torch.bincount(ids[(ids >= 0) & (ids < V)], minlength=V)[:, None].double()
    bound = (count.clamp(max=64) + count / 64 + 2) * 2.0 ** -24 * size
    bound = bound + (torch.finfo(out_dtype).eps / 2) * (want.abs() + bound)
    assert ((out - want).abs() <= bound).all()
    assert rlk.device_error() == 0


def test_a_tables_row_depends_on_its_own_rows_alone():
    n, V, H = 3000, 400, 72
    ids, d = some_ids(n, V, 6), numbers(n, H, seed=7)
    out = rlk.embedding_backward(d, ids, V, 1.0, FP32)
    for v in (V // 2, int(ids[ids >= 0][0])):
        mine = ids == v
        others = torch.where(mine, ids, (ids * 7 + 3) % V)
        others = torch.where(~mine & (others == v), -1, others)
        assert bits_equal(rlk.embedding_backward(d, others, V, 1.0, FP32)[v], out[v])
        alone = rlk.embedding_backward(d[mine], ids[mine], V, 1.0, FP32)
        assert bits_equal(alone[v], out[v])
    assert bits_equal(rlk.embedding_backward(d, ids, V, 1.0, FP32), out)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,V,H,pitch", [(500, 130, 50, 50), (90, 2100, 64, 72), (3, 9, 33, 35)])
def test_accumulation_leaves_other_rows_alone(n, V, H, pitch, dtype):
    ids, d = some_ids(n, V, 8), numbers(n, H, dtype=dtype, seed=9)
    table = numbers(V, pitch, dtype=FP32, seed=10)
    table[1, 0] = math.nan
    ids[ids == 1] = 0
    before = table.clone()
    back = rlk.embedding_grad_accum_fp32_(table[:, :H], d, ids, 0.5)
    assert back.data_ptr() == table.data_ptr()
    sums = rlk.embedding_backward(d, ids, V, 0.5, FP32)
    named = torch.zeros(V, dtype=torch.bool, device=ids.device)
    named[ids[(ids >= 0) & (ids < V)]] = True
    want = before.clone()
    want[named, :H] = before[named, :H] + sums[named]
    assert bits_equal(table, want)


def test_trainable():
    V, H = 300, 56
    ids = some_ids(40, V, 11).view(8, 5)
    for dtype in (BF16, FP32):
        w = numbers(V, H, dtype=dtype, seed=12).requires_grad_()
        d = numbers(8, 5, H, dtype=dtype, seed=13)
        out = rlk.embedding_trainable(ids, w, 2.5)
        assert bits_equal(out, rlk.embedding(ids, w.detach(), 2.5))
        grad, = torch.autograd.grad(out, w, d, retain_graph=True)
        assert grad.dtype == dtype and bits_equal(grad, rlk.embedding_backward(d, ids, V, 2.5, dtype))
        # a gradient that is one value, broadcast
        one, = torch.autograd.grad(out.sum(), w)
        assert bits_equal(one, rlk.embedding_backward(torch.ones_like(d), ids, V, 2.5, dtype))


def test_empty_and_refusals():
    w = numbers(10, 16)
    ids = some_ids(4, 10)
    d = numbers(4, 16)
    assert not rlk.embedding_backward(d[:0], ids[:0], 10).any()
    table = numbers(10, 16, dtype=FP32)
    keep = table.clone()
    assert torch.equal(rlk.embedding_grad_accum_fp32_(table, d[:0], ids[:0]), keep)
    with pytest.raises(TypeError):
        rlk.embedding(ids.int(), w)
    with pytest.raises(TypeError):
        rlk.embedding(ids, w.half())
    with pytest.raises(rlk.RlkError, match="RLK_ERR_VALUE"):
        rlk.embedding(ids, w, math.inf)
    with pytest.raises(RuntimeError, match="forward-only"):
        rlk.embedding(ids, w.requires_grad_())
    with pytest.raises(ValueError):
        rlk.embedding_backward(d, ids[:3], 10)
    with pytest.raises(rlk.RlkError, match="RLK_ERR_VALUE"):
        rlk.embedding_backward(d, ids, 10, math.nan)
    with pytest.raises(TypeError):
        rlk.embedding_grad_accum_fp32_(table.bfloat16(), d, ids)
    with pytest.raises(ValueError):
        rlk.embedding_grad_accum_fp32_(table.t(), numbers(4, 10), ids)
