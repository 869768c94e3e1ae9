"""A host thread's first CUDA call may be one of the library's: with its tensors from the allocator's
cache nothing before it has made the device's context current there (torch's autograd thread is such
a thread), and the tensor maps of the tensor-core kernels need one."""
import threading

import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
from helpers import bits_equal, cuda_or_skip

pytestmark = pytest.mark.gpu


def in_a_new_thread(call):
    got = []

    def run():
        try:
            got.append(call())
        except Exception as e:           # noqa: BLE001 (shown in the test's own thread)
            got.append(e)

    thread = threading.Thread(target=run)
    thread.start()
    thread.join()
    if isinstance(got[0], Exception):
        raise got[0]
    return got[0]


CALLS = {
    "det_gemm": lambda x, w: (rlk.det_gemm_fwd(x, w.t().contiguous()),),
    "det_linear_backward": lambda x, w: rlk.det_linear_backward(rlk.det_linear(x, w), x, w),
    "linear_logp": lambda x, w: rlk.linear_logp(x, w, torch.zeros(40, dtype=torch.int64, device=x.device)),
    "gated_linear": lambda x, w: (rlk.gated_linear(x, w),),
    "gated_linear_backward": lambda x, w: rlk.gated_linear_backward(rlk.gated_linear(x, w), x, w),
}


@pytest.mark.parametrize("name", CALLS)
def test_the_first_call_of_a_thread(name):
    dev = cuda_or_skip()
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn(40, 64, device=dev, generator=g).bfloat16()
    w = torch.randn(128, 64, device=dev, generator=g).bfloat16()
    want = CALLS[name](x, w)             # fills the allocator's cache and loads the kernels
    torch.cuda.synchronize()
    CALLS[name](x, w)
    torch.cuda.synchronize()
    got = in_a_new_thread(lambda: CALLS[name](x, w))
    torch.cuda.synchronize()
    assert all(bits_equal(a, b) for a, b in zip(got, want))
