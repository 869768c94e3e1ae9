"""Which kept logits the distillation backward reads in place, and that the others are copied into
rows of whole sectors whose every number may be read (CPU tensors: nothing is launched)."""
import pytest
import torch

from deterministic_invariant_gemm_linear_gb300 import _kept_logits


def readable(z, N, ld, V):
    """Every number the backward reads lies in z's storage."""
    last = z.storage_offset() + (N - 1) * ld + -(-V // 8) * 8
    return last * 4 <= z.untyped_storage().nbytes()


@pytest.mark.parametrize("N", [1, 2, 5])
@pytest.mark.parametrize("V", [1, 7, 8, 1001, 1008])
def test_any_layout(N, V):
    width = -(-V // 8) * 8
    own = torch.arange(N * width, dtype=torch.float32).view(N, width)[:, :V]
    wide = torch.zeros(N, width + 24)
    wide[:, 3:3 + V] = own
    column = own.t().contiguous().t()
    short = torch.empty(N * width + 16)[:(N - 1) * width + V].as_strided((N, V), (width, 1))
    short = short.clone(memory_format=torch.contiguous_format).copy_(own)
    layouts = {"own": own, "clone": own.clone(), "contiguous": own.contiguous().clone(),
               "shifted": wide[:, 3:3 + V], "columns": column, "short": short,
               "expanded": own[:1].expand(N, V)}
    for name, z in layouts.items():
        rows, ld = _kept_logits(z, N, V)
        assert rows.data_ptr() % 32 == 0 and ld % 8 == 0 and ld >= width, name
        assert readable(rows, N, ld, V), name
        got = rows.as_strided((N, V), (ld, 1), rows.storage_offset())
        assert torch.equal(got, z), name
    rows, ld = _kept_logits(own, N, V)
    assert rows.data_ptr() == own.data_ptr() and (N == 1 or ld == own.stride(0))


def test_last_row_of_a_buffer():
    """The last rows of a buffer with an odd vocabulary: no room for the last sector."""
    V = 1001
    base = torch.randn(3 * 1008 - 7)
    last = base[2 * 1008:].view(1, V)
    rows, ld = _kept_logits(last, 1, V)
    assert rows.data_ptr() != last.data_ptr() and ld == 1008 and torch.equal(rows[:, :V], last)
    both = base[1008:].as_strided((2, V), (1008, 1), 1008)
    rows, _ = _kept_logits(both, 2, V)
    assert rows.data_ptr() != both.data_ptr() and torch.equal(rows[:, :V], both)
