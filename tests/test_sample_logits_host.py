"""Refusals of the sampling entry point (no GPU needed: the fake addresses are never read)."""
import ctypes

import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk

P, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def lib():
    from deterministic_invariant_gemm_linear_gb300 import build as b
    b.build()
    return rlk.lib()


CALL = dict(logits=P, dt=1, N=4, V=10, ld=10, u=P, ut=2, tau=None, tau_all=1.0, k=None, k_all=0,
            p=None, p_all=1.0, m=None, m_all=0.0, token=P, logp=P, ws=None, n=0, stream=None)
NAN = float("nan")


@pytest.mark.parametrize("change,status", [
    (dict(N=-1), 2), (dict(N=1 << 20), 2), (dict(V=0, ld=0), 2), (dict(V=524289, ld=524289), 2),
    (dict(ld=9), 2), (dict(dt=2), 3), (dict(dt=-1), 3), (dict(ut=0), 3), (dict(ut=3), 3),
    (dict(tau_all=-1.0), 11), (dict(tau_all=NAN), 11), (dict(tau_all=float("inf")), 11),
    (dict(p_all=NAN), 11), (dict(m_all=NAN), 11), (dict(logits=None), 1), (dict(u=None), 1),
    (dict(token=None), 1), (dict(logp=None), 1), (dict(logits=ODD), 4), (dict(u=ODD), 4),
    (dict(u=ctypes.c_void_p(0x10004)), 4), (dict(tau=ODD), 4), (dict(k=ODD), 4), (dict(p=ODD), 4),
    (dict(m=ODD), 4), (dict(token=ctypes.c_void_p(0x10004)), 4), (dict(logp=ODD), 4)])
def test_refusals(lib, change, status):
    assert lib.rlk_sample_logits(*{**CALL, **change}.values()) == status


def test_workspace(lib):
    f = lib.rlk_sample_logits_workspace_size
    assert f(1, 1, 151936) == 0 and f(0, 64, 32003) == 0
    N, V = 1024, 151936
    tiles = -(-(-(-(V + 3) // 4)) // 256)
    up = lambda x: -(-x // 256) * 256
    assert f(1, N, V) == up(N * tiles * 128) + up(N * tiles * 8) + N * 8192 + N * 40 + up(N * 4 + 4) + N * 16384
    assert f(2, N, V) == 0 and f(1, -1, V) == 0 and f(1, N, 0) == 0 and f(1, N, 524289) == 0
    big = {**CALL, "N": N, "V": V, "ld": V}
    assert lib.rlk_sample_logits(*big.values()) == 5
    assert lib.rlk_sample_logits(*{**big, "ws": P, "n": 1000}.values()) == 5
    assert lib.rlk_sample_logits(*{**big, "ws": ctypes.c_void_p(0x10010), "n": 1 << 30}.values()) == 5


def test_no_rows_need_no_device(lib):
    assert lib.rlk_sample_logits(*{**CALL, "N": 0, "logits": None}.values()) == 0


def test_python_refusals(lib):
    with pytest.raises(ValueError, match="CUDA"):
        rlk.sample_logits(torch.zeros(2, 8), torch.zeros(2))
