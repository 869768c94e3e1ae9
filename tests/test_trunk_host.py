"""Refusals and workspace sizes of the trunk's entry points (no GPU needed: the fake addresses are
never read, every call fails validation first)."""
import ctypes

import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk

P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)
HALF = ctypes.c_void_p(0x10002)
NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, VALUE = 1, 2, 3, 4, 5, 11
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from deterministic_invariant_gemm_linear_gb300 import build as b
    b.build()
    return rlk.lib()


def up(x, a=256):
    return -(-x // a) * a


EMBED = dict(ids=P, step=1, N=4, weight=P, wdt=0, V=10, H=8, ldw=8, scale=1.0, out=P, odt=0, ldo=8, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(N=-1), SHAPE), (dict(N=1 << 31), SHAPE), (dict(V=0), SHAPE), (dict(V=1 << 31), SHAPE), (dict(H=0), SHAPE),
    (dict(H=1 << 20, ldw=1 << 20, ldo=1 << 20), SHAPE), (dict(step=-1), SHAPE), (dict(ldw=7), SHAPE),
    (dict(ldo=7), SHAPE), (dict(wdt=2), DTYPE), (dict(odt=-1), DTYPE), (dict(scale=NAN), VALUE),
    (dict(scale=-INF), VALUE), (dict(ids=None), NULL), (dict(weight=None), NULL), (dict(out=None), NULL),
    (dict(ids=HALF), ALIGN), (dict(weight=ODD), ALIGN), (dict(out=ODD), ALIGN), (dict(weight=HALF, wdt=1), ALIGN),
    (dict(out=HALF, odt=1), ALIGN), (dict(N=0, ids=None, weight=None, out=None), 0)])
def test_embedding(lib, change, status):
    assert lib.rlk_embedding(*{**EMBED, **change}.values()) == status


EGRAD = dict(ids=P, step=1, N=4, grad=P, gdt=0, H=8, ldg=8, scale=1.0, out=P, odt=1, V=10, ldo=8, acc=0, ws=P,
             n=1 << 20, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(N=-1), SHAPE), (dict(V=0), SHAPE), (dict(V=1 << 30), SHAPE), (dict(H=0), SHAPE), (dict(step=-1), SHAPE),
    (dict(N=1 << 21, V=1 << 26), SHAPE), (dict(ldg=7), SHAPE), (dict(ldo=7), SHAPE), (dict(gdt=2), DTYPE), (dict(odt=2), DTYPE),
    (dict(odt=0, acc=1), DTYPE), (dict(scale=INF), VALUE), (dict(ids=None), NULL), (dict(grad=None), NULL),
    (dict(out=None), NULL), (dict(ids=HALF), ALIGN), (dict(grad=ODD), ALIGN), (dict(out=HALF), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(ws=ctypes.c_void_p(0x10010)), WORKSPACE), (dict(n=100), WORKSPACE),
    (dict(N=0, acc=1, ids=None, grad=None, ws=None), 0)])
def test_embedding_backward(lib, change, status):
    assert lib.rlk_embedding_backward(*{**EGRAD, **change}.values()) == status


def test_embedding_workspace(lib):
    size = lib.rlk_embedding_backward_workspace_size
    # offsets, rows, groups, counts of them, their sums: an id of c > 64 rows makes ceil(c / 64)
    for N, V, H in ((1, 1, 1), (64, 10, 8), (65, 10, 9), (16384, 151936, 4096)):
        groups = 2 * N // 65
        assert size(N, V, H) == up(4 * (V + 1)) + up(4 * N) + up(16 * groups) + \
            up(groups * -(-H // 2048) * 4) + up(groups * up(H, 8) * 4)
        worst = max((N // c) * -(-c // 64) for c in range(65, min(N, 400) + 1)) if N > 64 else 0
        assert worst <= groups
    assert size(-1, 10, 8) == 0 and size(4, 0, 8) == 0 and size(4, 10, 0) == 0 and size(4, 1 << 30, 8) == 0


def test_first_groups_leave_room():
    """An id of c > 64 rows from place p on has its ceil(c / 64) groups from 2 p // 65 on: before the
    next id's, whatever p."""
    for c in list(range(65, 2000)) + [10 ** 4, 10 ** 5 + 1, 2 ** 20, 2 ** 30 + 7]:
        for p in (0, 1, 31, 32, 33, 64, 65, 1000, 2 ** 30):
            assert 2 * p // 65 + -(-c // 64) <= 2 * (p + c) // 65


PACK = dict(x=P, dt=0, rows=4, cols=40, ldx=40, q=P, ldq=64, e=P, lde=2, stream=None)
UNPACK = dict(q=P, rows=4, cols=40, ldq=64, e=P, lde=2, out=P, dt=0, ldo=40, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(cols=1 << 30), SHAPE), (dict(ldq=48), SHAPE),
    (dict(ldq=72), SHAPE), (dict(lde=1), SHAPE), (dict(dt=2), DTYPE), (dict(q=None), NULL), (dict(e=None), NULL),
    (dict(q=ctypes.c_void_p(0x10008)), ALIGN), (dict(rows=0, q=None, e=None), 0)])
def test_int8(lib, change, status):
    assert lib.rlk_pack_int8(*{**PACK, **change}.values()) == status
    assert lib.rlk_unpack_int8(*{**UNPACK, **change}.values()) == status


@pytest.mark.parametrize("change,status", [(dict(ldx=39), SHAPE), (dict(x=None), NULL), (dict(x=ODD), ALIGN),
                                           (dict(x=HALF, dt=1), ALIGN)])
def test_pack_int8(lib, change, status):
    assert lib.rlk_pack_int8(*{**PACK, **change}.values()) == status
    other = {"out" if k == "x" else "ldo" if k == "ldx" else k: v for k, v in change.items()}
    assert lib.rlk_unpack_int8(*{**UNPACK, **other}.values()) == status


GATED = dict(X=P, M=4, K=8, ldx=8, W=P, F=10, ldw=8, act=0, H=P, hdt=0, ldh=10, keep=0, kept=None, e=None, ws=P,
             n=1 << 20, stream=None)
GGRAD = dict(dH=P, ddt=0, M=4, F=10, ldd=10, X=P, K=8, ldx=8, W=P, ldw=8, act=0, keep=0, kept=None, e=None, dX=P,
             dxt=0, lddx=8, dW=P, dwt=0, lddw=8, ws=P, n=1 << 20, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(K=0), SHAPE), (dict(K=1 << 20, ldx=1 << 20, ldw=1 << 20), SHAPE),
    (dict(F=0), SHAPE), (dict(F=1 << 30), SHAPE), (dict(ldx=7), SHAPE), (dict(ldw=7), SHAPE), (dict(act=2), VALUE),
    (dict(act=-1), VALUE), (dict(keep=3), VALUE), (dict(keep=-1), VALUE), (dict(X=None), NULL), (dict(W=None), NULL),
    (dict(X=ODD), ALIGN), (dict(W=ODD), ALIGN), (dict(keep=1), NULL), (dict(keep=2, kept=P), NULL),
    (dict(keep=1, kept=ctypes.c_void_p(0x10010)), ALIGN), (dict(ws=None), WORKSPACE),
    (dict(ws=ctypes.c_void_p(0x10010)), WORKSPACE), (dict(n=255), WORKSPACE)])
def test_gated_linear(lib, change, status):
    assert lib.rlk_gated_linear(*{**GATED, **change}.values()) == status
    if not ("F" in change and change["F"] > 10):       # the other pitches stay those of F = 10
        assert lib.rlk_gated_linear_backward(*{**GGRAD, **change}.values()) == status


@pytest.mark.parametrize("change,status", [(dict(H=None), NULL), (dict(H=ODD), ALIGN), (dict(H=HALF, hdt=1), ALIGN),
                                           (dict(ldh=9), SHAPE), (dict(hdt=2), DTYPE),
                                           (dict(M=0, X=None, W=None, H=None, ws=None), 0)])
def test_gated_linear_forward(lib, change, status):
    assert lib.rlk_gated_linear(*{**GATED, **change}.values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(dH=None), NULL), (dict(dH=ODD), ALIGN), (dict(dH=HALF, ddt=1), ALIGN), (dict(ldd=9), SHAPE),
    (dict(ddt=2), DTYPE), (dict(dX=ODD), ALIGN), (dict(dW=HALF, dwt=1), ALIGN), (dict(lddx=7), SHAPE),
    (dict(lddw=7), SHAPE), (dict(dxt=2), DTYPE), (dict(dwt=-1), DTYPE), (dict(dX=None, dW=None, X=None, W=None), 0),
    (dict(keep=1, kept=P, X=None), NULL), (dict(keep=1, kept=P, W=None), NULL), (dict(X=None, dW=None), NULL),
    (dict(M=0, dW=None, ws=None), 0)])
def test_gated_linear_backward(lib, change, status):
    assert lib.rlk_gated_linear_backward(*{**GGRAD, **change}.values()) == status


def test_gated_workspaces(lib):
    f, b = lib.rlk_gated_linear_workspace_size, lib.rlk_gated_linear_backward_workspace_size
    M, K, F = 300, 64, 1001
    assert f(P, M, K, K, P, F, K) == 256
    assert b(P, M, K, K, P, F, K) == up(M * up(2 * F, 8) * 2) + 256
    for size in (f, b):
        base = size(P, M, K, K, P, F, K)
        assert size(P, M, K, 65, P, F, K) - base == up(M * 64 * 2)
        assert size(HALF, M, K, K, P, F, 67) - base == up(M * 64 * 2) + up(2 * F * 64 * 2)
        assert size(P, M, 0, K, P, F, K) == size(P, -1, K, K, P, F, K) == size(P, M, K, K, P, 0, K) == 0


def test_python_refusals(lib):
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    ids = torch.zeros(2, dtype=torch.int64)
    for call in (lambda: rlk.embedding(ids, x), lambda: rlk.embedding_backward(x, ids, 4), lambda: rlk.pack_int8(x),
                 lambda: rlk.unpack_int8(x.to(torch.int8), x.to(torch.uint8)), lambda: rlk.gated_linear(x, x),
                 lambda: rlk.gated_linear_backward(x, x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
