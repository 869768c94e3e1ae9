"""Nothing outside the outputs and the stated workspace is written: each is laid between guard
bands, at its exact size, through the C ABI."""
import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
from helpers import cuda_or_skip

pytestmark = pytest.mark.gpu
BAND, FILL = 4096, 0xA5


class Guarded:
    """Device buffers of exact sizes, each between two bands of a fixed byte."""

    def __init__(self, dev):
        self.dev, self.held = dev, []

    def take(self, nbytes, dtype=torch.uint8, shape=None):
        raw = torch.full((2 * BAND + -(-nbytes // 256) * 256,), FILL, dtype=torch.uint8, device=self.dev)
        self.held.append((raw, nbytes))
        view = raw[BAND:BAND + nbytes]
        return view if shape is None else view.view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        assert rlk.device_error() == 0
        for raw, n in self.held:
            assert (raw[:BAND] == FILL).all() and (raw[BAND + n:] == FILL).all()


@pytest.mark.parametrize("N,V,dtype", [(1, 1, torch.float32), (3, 1001, torch.bfloat16),
                                       (70, 20011, torch.float32), (130, 16385, torch.bfloat16),
                                       (110, 20011, torch.float32), (270, 16385, torch.bfloat16)])
@pytest.mark.parametrize("k,p,m", [(0, 1.0, 0.0), (40, 0.9, 0.0), (0, 0.9, 0.01), (3000, 0.9, 0.0)])
def test_sampling(N, V, dtype, k, p, m):
    dev = cuda_or_skip()
    g = torch.Generator(device=dev).manual_seed(N)
    z = (torch.randn(N, V, device=dev, generator=g) * 2).to(dtype)
    z[::3] *= 0.2
    u = torch.rand(N, device=dev, generator=g, dtype=torch.float64)
    b = Guarded(dev)
    lib = rlk.lib()
    n = lib.rlk_sample_logits_workspace_size(rlk._DT[dtype], N, V)
    assert (n > 0) == (V >= 16384 and N * V * z.element_size() >= 8 << 20)
    ws = b.take(n)
    token = b.take(8 * N, torch.int64, (N,))
    logp = b.take(4 * N, torch.float32, (N,))
    st = lib.rlk_sample_logits(z.data_ptr(), rlk._DT[dtype], N, V, V, u.data_ptr(), rlk.RLK_FP64, None,
                               0.9, None, k, None, p, None, m, token.data_ptr(), logp.data_ptr(),
                               ws.data_ptr() if n else None, n, rlk._stream_ptr(None))
    assert st == 0
    b.check()
    want = rlk.sample_logits(z, u, temperature=0.9, top_k=k, top_p=p, min_p=m)
    assert torch.equal(token, want[0]) and torch.equal(logp, want[1])


@pytest.mark.parametrize("N,H,V,K", [(1, 1, 1, 1), (17, 40, 301, 5), (130, 33, 1030, 64), (300, 72, 515, 9)])
@pytest.mark.parametrize("kept", [False, True])
def test_distillation(N, H, V, K, kept):
    dev = cuda_or_skip()
    g = torch.Generator(device=dev).manual_seed(V)
    h = torch.randn(N, H, device=dev, generator=g).bfloat16()
    w = torch.randn(V, H, device=dev, generator=g).bfloat16()
    bias = torch.randn(V, device=dev, generator=g)
    ids = torch.randint(V, (N, K), device=dev, generator=g)
    t = torch.randn(N, K, device=dev, generator=g)
    up = torch.randn(N, device=dev, generator=g)
    b, lib = Guarded(dev), rlk.lib()
    operands = (h.data_ptr(), N, H, H, w.data_ptr(), V, H)
    teacher = (bias.data_ptr(), ids.data_ptr(), K, t.data_ptr(), rlk.RLK_FP32, K, K, None, 1.5)
    n = lib.rlk_linear_distill_workspace_size(*operands, K)
    ws = b.take(n)
    loss, lse = (b.take(4 * N, torch.float32, (N,)) for _ in range(2))
    ldz = -(-V // 8) * 8
    z = b.take(4 * N * ldz, torch.float32, (N, ldz)) if kept else None
    zp = z.data_ptr() if kept else None
    assert lib.rlk_linear_distill(*operands, *teacher, loss.data_ptr(), lse.data_ptr(), zp, ldz,
                                  ws.data_ptr(), n, rlk._stream_ptr(None)) == 0
    b.check()
    n = lib.rlk_linear_distill_backward_workspace_size(*operands, K, 1)
    ws = b.take(n)
    gh, gw = b.take(2 * N * H, torch.bfloat16, (N, H)), b.take(2 * V * H, torch.bfloat16, (V, H))
    gb = b.take(4 * V, torch.float32, (V,))
    assert lib.rlk_linear_distill_backward(
        *operands, *teacher, lse.data_ptr(), zp, ldz, up.data_ptr(), gh.data_ptr(), 0, H, gw.data_ptr(),
        0, H, gb.data_ptr(), ws.data_ptr(), n, rlk._stream_ptr(None)) == 0
    b.check()
    want = rlk.linear_distill_backward(h, w, ids, t, lse, up, bias, temperature=1.5)
    assert torch.equal(gh, want[0]) and torch.equal(gw, want[1]) and torch.equal(gb, want[2])
