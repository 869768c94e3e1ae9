"""Both products of the gated block's backward in one launch, with either of them the longer."""
import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
from helpers import bits_equal, cuda_or_skip

pytestmark = pytest.mark.gpu
FP32 = torch.float32
PAIR_ROWS, TILE, STAGE = 256, 256, 64


def in_one_launch(M, K, F, pairs):
    """The rule of rlk_gated_linear_backward for one launch over both tile lists."""
    longer, shorter = max(M, 2 * F), min(M, 2 * F)
    across = -(-K // TILE)
    short_tiles = -(-longer // PAIR_ROWS) * across
    if 2 * -(-shorter // PAIR_ROWS) * across > pairs or short_tiles < 8 * pairs:
        return False
    return 100 * short_tiles * (-(-shorter // STAGE) + 6) > 45 * pairs * -(-longer // STAGE)


# whose reduction is the longer: grad X's over 2 F, grad W's over the rows
@pytest.mark.parametrize("M,K,F", [(255, 4096, 6000), (37, 6144, 4856), (9001, 4355, 125), (17000, 4848, 90)])
def test_one_launch_has_the_bits_of_two(M, K, F):
    dev = cuda_or_skip()
    assert in_one_launch(M, K, F, torch.cuda.get_device_properties(dev).multi_processor_count // 2)
    g = torch.Generator(device=dev).manual_seed(M + F)
    x = torch.randn(M, K, device=dev, generator=g).bfloat16()
    w = (torch.randn(2 * F, K, device=dev, generator=g) / K ** 0.5).bfloat16()
    d = torch.randn(M, F, device=dev, generator=g).bfloat16()
    kept = rlk.gated_linear(x, w, keep="int8")[1]
    for held in (None, kept):
        for dtype in (torch.bfloat16, FP32):
            gx, gw, G = rlk.gated_linear_backward(d, x, w, kept=held, out_dtype=dtype, return_grad_projections=True)
            one, two = rlk.det_linear_dx(G.contiguous(), w, dtype), rlk.det_linear_dw(G.contiguous(), x, dtype)
            assert bits_equal(gx, one) and bits_equal(gw, two)
            # FP32 sums of `red` products, 16 an addition, each off by at most 2^-23 of a partial sum
            if dtype == FP32:
                want = (G.double() @ w.double(), 2 * F), (G.double().t() @ x.double(), M)
                for a, (b, red) in zip((gx, gw), want):
                    assert (a.double() - b).norm() <= (red / 16 + 2) * 2.0 ** -23 * b.norm()
    assert rlk.device_error() == 0
