"""The temperatures that distillation takes: past 100, T^2 times the error of an FP32 sum is as large
as the loss (no GPU needed: the fake addresses are never read)."""
import math

import pytest

from test_linear_distill_host import BWD, FWD, lib  # noqa: F401


@pytest.mark.parametrize("T", [100.5, 1e3, 1e4, 9e-5, -0.0])
def test_refused(lib, T):  # noqa: F811
    assert lib.rlk_linear_distill(*{**FWD, "T": T}.values()) == 11
    assert lib.rlk_linear_distill_backward(*{**BWD, "T": T}.values()) == 11


@pytest.mark.parametrize("T", [100.0, 1e-4 * (1 + 2 ** -20), math.pi])
def test_taken(lib, T):  # noqa: F811
    """Refused for the missing workspace, after the temperature was taken."""
    assert lib.rlk_linear_distill(*{**FWD, "T": T, "ws": None}.values()) == 5
    assert lib.rlk_linear_distill_backward(*{**BWD, "T": T, "ws": None}.values()) == 5
