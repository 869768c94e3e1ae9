"""Refusals and workspace sizes of the distillation entry points (no GPU needed: the fake
addresses are never read, every call fails validation first)."""
import ctypes

import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk

P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def lib():
    from deterministic_invariant_gemm_linear_gb300 import build as b
    b.build()
    return rlk.lib()


FWD = dict(hidden=P, N=4, H=8, ldh=8, weight=P, V=10, ldw=8, bias=None, ids=P, ldi=3, tl=P, dt=1,
           ldt=3, K=3, tlse=None, T=1.0, loss=P, lse=P, z=None, ldz=0, ws=P, n=1 << 20, stream=None)
BWD = dict(hidden=P, N=4, H=8, ldh=8, weight=P, V=10, ldw=8, bias=None, ids=P, ldi=3, tl=P, dt=1,
           ldt=3, K=3, tlse=None, T=1.0, lse=P, z=None, ldz=0, grad=P, gh=P, ghd=0, ldgh=8, gw=P, gwd=0, ldgw=8,
           gb=None, ws=P, n=1 << 20, stream=None)

REFUSALS = [
    (dict(N=-1), 2), (dict(H=0), 2), (dict(V=0), 2), (dict(ldh=7), 2), (dict(ldw=7), 2),
    (dict(K=-1), 2), (dict(K=4), 2), (dict(K=1025, ldi=1025, ldt=1025), 2), (dict(ldi=2), 2),
    (dict(ldt=2), 2), (dict(dt=2), 3), (dict(T=0.0), 11), (dict(T=-1.0), 11),
    (dict(T=float("nan")), 11), (dict(T=float("inf")), 11), (dict(hidden=None), 1),
    (dict(weight=None), 1), (dict(ids=None), 1), (dict(tl=None), 1), (dict(lse=None), 1),
    (dict(hidden=ODD), 4), (dict(weight=ODD), 4), (dict(bias=ODD), 4), (dict(ids=ODD), 4),
    (dict(tl=ODD), 4), (dict(tlse=ODD), 4), (dict(lse=ODD), 4), (dict(ws=None), 5), (dict(n=64), 5),
    (dict(ws=ctypes.c_void_p(0x10010)), 5), (dict(z=P, ldz=12), 2), (dict(z=P, ldz=8), 2),
    (dict(z=ctypes.c_void_p(0x10010), ldz=16), 4),
]


@pytest.mark.parametrize("change,status", REFUSALS)
def test_refusals_of_both(lib, change, status):
    assert lib.rlk_linear_distill(*{**FWD, **change}.values()) == status
    assert lib.rlk_linear_distill_backward(*{**BWD, **change}.values()) == status


@pytest.mark.parametrize("change,status", [(dict(loss=None), 1), (dict(loss=ODD), 4)])
def test_refusals_of_the_forward(lib, change, status):
    assert lib.rlk_linear_distill(*{**FWD, **change}.values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(grad=None), 1), (dict(grad=ODD), 4), (dict(gh=ODD), 4), (dict(gw=ODD), 4), (dict(gb=ODD), 4),
    (dict(ldgh=7), 2), (dict(ldgw=7), 2), (dict(ghd=2), 3), (dict(gwd=-1), 3),
    (dict(ghd=1, gh=ctypes.c_void_p(0x10002)), 4)])
def test_refusals_of_the_backward(lib, change, status):
    assert lib.rlk_linear_distill_backward(*{**BWD, **change}.values()) == status


def test_empty_calls_need_no_device(lib):
    assert lib.rlk_linear_distill(*{**FWD, "N": 0}.values()) == 0
    assert lib.rlk_linear_distill_backward(*{**BWD, "N": 0, "gw": None}.values()) == 0


def up(x, a=256):
    return -(-x // a) * a


def test_workspace_sizes(lib):
    f, b = lib.rlk_linear_distill_workspace_size, lib.rlk_linear_distill_backward_workspace_size
    N, H, V, K = 300, 64, 1000, 20
    S = 4
    lists = 2 * up(N * K * 4) + up(N * (S + 1) * 2) + up(N * 8)
    assert f(P, N, H, H, P, V, H, K) == up(N * S * 8) + up(N * S * 4) + 256 + lists
    assert b(P, N, H, H, P, V, H, K, 0) == up(N * V * 2) + 256 + lists
    assert b(P, N, H, H, P, V, H, K, 1) == up(N * V * 2) + up(10 * V * 4) + 256 + lists
    assert f(P, N, H, 65, P, V, H, K) - f(P, N, H, H, P, V, H, K) == up(N * 64 * 2)
    for bad in ((P, -1, H, H, P, V, H, K), (P, N, 0, H, P, V, H, K), (P, N, H, 63, P, V, H, K),
                (P, N, H, H, P, V, H, 1025), (P, N, H, H, P, V, H, -1)):
        assert f(*bad) == 0 and b(*bad, 0) == 0


def test_python_refusals(lib):
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    ids = torch.zeros(2, 3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        rlk.linear_distill(x, x, ids, torch.zeros(2, 3))
