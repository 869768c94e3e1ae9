"""The table gradient of nearly as many rows as a call takes, all of one id."""
import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
from helpers import cuda_or_skip

pytestmark = pytest.mark.gpu


def test_as_many_rows_of_one_id_as_there_can_be():
    """Past 2^31 - 65536 rows of one id the row numbers behind its last group leave 32 bits."""
    dev = cuda_or_skip()
    if torch.cuda.mem_get_info(dev)[0] < 32 << 30:
        pytest.skip("needs 32 GB on the device")
    N = 2 ** 31 - 300
    ids = torch.ones(1, dtype=torch.int64, device=dev).expand(N)
    grad = torch.zeros(N, 1, dtype=torch.bfloat16, device=dev)
    # one bit of the sum from each of these rows: exact in FP32, whatever the order
    rows = [0, 63, 64, 65_535, 2 ** 30, 2 ** 30 + 64, 2 ** 31 - 65_536, 2 ** 31 - 65_537, N - 45, N - 1]
    for k, r in enumerate(rows):
        grad[r] = 2.0 ** k
    out = rlk.embedding_backward(grad, ids, 3, 0.5, torch.float32)
    assert out[:, 0].tolist() == [0.0, 0.5 * (2.0 ** len(rows) - 1), 0.0]
    assert rlk.device_error() == 0
