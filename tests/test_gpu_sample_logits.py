"""Sampling on the GPU: tokens equal to the definition's, id by id, log-probabilities against
64 bits, refusals of rows without a distribution, and what must not change a token."""
import math

import numpy as np
import pytest
import torch

import deterministic_invariant_gemm_linear_gb300 as rlk
import sample_reference as ref
from helpers import bits_equal, cuda_or_skip

pytestmark = pytest.mark.gpu

SETTINGS = [dict(), dict(temperature=0.0), dict(temperature=0.7, top_k=50), dict(top_p=0.9),
            dict(min_p=0.05), dict(temperature=1.3, top_k=20, top_p=0.8, min_p=0.02),
            dict(top_k=1), dict(top_p=0.0), dict(min_p=1.0), dict(temperature=1e-4, top_p=0.99)]


def logits(N, V, seed, spread=2.0, peak=True):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(N, V, generator=g) * spread
    if peak:
        at = torch.randint(V, (N, max(1, min(V, 20))), generator=g)
        z.scatter_add_(1, at, torch.rand(at.shape, generator=g) * 12)
    return z


def check(dev, z, u, stream=None, **how):
    """Runs the rows and compares every token with the reference's."""
    def put(x):
        return x.to(dev) if torch.is_tensor(x) else x
    zd = z if z.is_cuda else z.to(dev)
    token, logp = rlk.sample_logits(zd, u.to(dev), **{k: put(v) for k, v in how.items()})
    assert rlk.device_error() == 0
    zf = zd.float().cpu().numpy()
    plain = {k: v.numpy() if torch.is_tensor(v) else v for k, v in how.items()}
    want, want_logp = ref.rows(zf, u.double().numpy(), **plain)
    assert np.array_equal(token.cpu().numpy(), want), (token.cpu().numpy() != want).nonzero()
    got = logp.cpu().double().numpy()
    ok = want >= 0
    assert np.isnan(got[~ok]).all()
    finite = np.where(np.isfinite(zf), zf, 0)
    spread = float(np.abs(finite).max()) * 2
    tau = np.broadcast_to(np.asarray(plain.get("temperature", 1.0), np.float64), want.shape)
    tau = np.where(tau < 1e-6, 1.0, tau)
    bound = [ref.logp_bound(l, zf.shape[1], spread, t) for l, t in zip(want_logp[ok], tau[ok])]
    assert (np.abs(got[ok] - want_logp[ok]) <= np.array(bound)).all()
    return token, logp


def uniforms(N, seed, dtype=torch.float64):
    return torch.rand(N, generator=torch.Generator().manual_seed(seed), dtype=dtype)


@pytest.mark.parametrize("how", SETTINGS)
@pytest.mark.parametrize("N,V", [(1, 1), (5, 2), (9, 33), (40, 1000), (3, 4099), (70, 5003), (6, 32003)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens(N, V, dtype, how):
    dev = cuda_or_skip()
    check(dev, logits(N, V, N * V).to(dtype), uniforms(N, V), **how)


@pytest.mark.parametrize("N,V,dtype", [(1, 151936, torch.float32), (5, 152064, torch.float32),
                                       (9, 100003, torch.bfloat16), (20, 152064, torch.bfloat16),
                                       (40, 151936, torch.float32), (2, 524288, torch.float32),
                                       (30, 70001, torch.float32), (160, 20011, torch.bfloat16),
                                       (48, 151936, torch.float32), (90, 152064, torch.bfloat16)])
@pytest.mark.parametrize("how", [dict(), dict(top_k=50, top_p=0.95), dict(top_p=0.9)])
def test_large_vocabularies(N, V, dtype, how):
    dev = cuda_or_skip()
    check(dev, logits(N, V, V).to(dtype), uniforms(N, 2), **how)


def kinds(N, V, seed):
    """Rows of every sort: confident, open, flat, equal, few levels, mostly banned, steep, broken."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(N, V, generator=g) * 2
    for r in range(N):
        kind = r % 11
        if kind == 0:
            z[r, torch.randint(V, (30,), generator=g)] += torch.rand(30, generator=g) * 14
        elif kind == 1:
            z[r] *= 0.3
        elif kind == 2:
            z[r] = 1.5
        elif kind == 3:
            z[r] = torch.randint(4, (V,), generator=g).float()
        elif kind == 4:
            z[r, torch.rand(V, generator=g) < 0.999] = -math.inf
        elif kind == 5:
            z[r] = -torch.linspace(0, 300, V)
        elif kind == 6:
            z[r, torch.rand(V, generator=g) < 0.5] = torch.finfo(torch.float32).min
        elif kind == 7:
            z[r, V // 2] = 40
        elif kind == 8:
            z[r, 0], z[r, V - 1] = 9, 9
        elif kind == 9 and r % 2:
            z[r, (r * 37) % V] = (math.nan, math.inf, -math.inf)[r % 3]
    return z


@pytest.mark.parametrize("N,V,dtype,shift", [(120, 20011, torch.float32, 0), (160, 16384, torch.bfloat16, 0),
                                             (60, 40007, torch.float32, 3), (110, 40009, torch.bfloat16, 5),
                                             (272, 16384, torch.bfloat16, 0)])
def test_many_rows(N, V, dtype, shift):
    """Calls large enough for the streaming kernels: rows of every sort, settings of every sort, and
    each row's token and bits those of a call of its own."""
    dev = cuda_or_skip()
    wide = torch.full((N, V + 13 if shift else V), 99.0, dtype=dtype, device=dev)
    z = wide[:, shift:shift + V]
    z.copy_(kinds(N, V, V).to(dtype))
    u = uniforms(N, 22)
    g = torch.Generator().manual_seed(23)
    def pick(v, dtype):
        return torch.tensor(v, dtype=dtype)[torch.randint(len(v), (N,), generator=g)]
    settings = [dict(), dict(top_k=40, top_p=0.9), dict(top_p=0.95), dict(top_p=0.5, min_p=0.01), dict(min_p=0.2),
                dict(temperature=0.0), dict(top_k=1000), dict(top_k=9000, top_p=0.97),
                dict(temperature=pick([0.0, 0.5, 1.0, 3.0], torch.float32),
                     top_k=pick([0, 0, 1, 50, 900, 3000, V - 1], torch.int32),
                     top_p=pick([0.2, 0.9, 0.999, 1.0, 1.0], torch.float32),
                     min_p=pick([0.0, 0.0, 0.001, 0.3], torch.float32))]
    nb = rlk.lib().rlk_sample_logits_workspace_size(rlk._DT[dtype], N, V)
    assert (nb > 0) == (N * V * z.element_size() >= 8 << 20)
    for how in settings:
        token, logp = check(dev, z, u, **how)
        for s in (slice(0, 9), slice(40, 75), slice(N - 12, N)):
            part = {k: v[s].to(dev) if torch.is_tensor(v) else v for k, v in how.items()}
            a = rlk.sample_logits(z[s], u[s].to(dev), **part)
            assert torch.equal(a[0], token[s]) and bits_equal(a[1], logp[s])


def test_settings_per_row():
    dev = cuda_or_skip()
    N = 200
    g = torch.Generator().manual_seed(3)
    def pick(v, dtype):
        return torch.tensor(v, dtype=dtype)[torch.randint(len(v), (N,), generator=g)]
    check(dev, logits(N, 3001, 4), uniforms(N, 5, torch.float32),
          temperature=pick([0.0, 0.5, 1.0, 2.0], torch.float32),
          top_k=pick([-1, 0, 1, 7, 100, 2999, 3001, 5000], torch.int32),
          top_p=pick([0.0, 0.3, 0.9, 0.999, 1.0, 1.5], torch.float32),
          min_p=pick([-0.5, 0.0, 0.01, 0.5, 1.0, 2.0], torch.float32))


@pytest.mark.parametrize("V", [3000, 60000])
@pytest.mark.parametrize("how", [dict(top_k=2500), dict(top_p=0.97), dict(top_k=2800, top_p=0.99),
                                 dict(top_p=0.999, min_p=1e-4), dict(top_k=2999, top_p=0.5)])
def test_cuts_past_the_candidate_list(V, how):
    """Open distributions, whose kept sets are larger than what one CTA sorts."""
    dev = cuda_or_skip()
    check(dev, logits(24, V, 6, 0.7, False), uniforms(24, 7), **how)
    check(dev, logits(24, V, 6, 0.7, False).bfloat16(), uniforms(24, 7), **how)


@pytest.mark.parametrize("V", [1, 31, 700, 9000, 40000])
@pytest.mark.parametrize("how", [dict(), dict(top_k=300), dict(top_p=0.4), dict(top_k=5000, top_p=0.77),
                                 dict(temperature=0.0)])
def test_equal_logits(V, how):
    """Cuts among equal logits go by id: constant rows, two values, and a few levels."""
    dev = cuda_or_skip()
    g = torch.Generator().manual_seed(8)
    z = torch.stack([torch.zeros(V), torch.full((V,), -7.25),
                     (torch.rand(V, generator=g) < 0.5).float(),
                     torch.randint(5, (V,), generator=g).float() * 0.5,
                     torch.where(torch.rand(V, generator=g) < 0.5, 0.0, -0.0)])
    check(dev, z, uniforms(5, 9), **how)


@pytest.mark.parametrize("how", [dict(), dict(top_k=10), dict(top_k=64, top_p=0.9), dict(min_p=0.1)])
@pytest.mark.parametrize("low", [-math.inf, float(torch.finfo(torch.float32).min), -1e30])
def test_banned_ids(how, low):
    """Few ids allowed out of many, whatever value bans the others."""
    dev = cuda_or_skip()
    z = torch.full((8, 20000), low)
    g = torch.Generator().manual_seed(10)
    for r in range(8):
        at = torch.randperm(20000, generator=g)[:1 + 5 * r]
        z[r, at] = torch.randn(len(at), generator=g) * 3
    token, _ = check(dev, z, uniforms(8, 11), **how)
    assert (z[torch.arange(8), token.cpu()] > -100).all()


def test_weights_that_vanish():
    """Logits 20 to 200 below the largest: cuts by count that fall among weights of 0."""
    dev = cuda_or_skip()
    z = -torch.linspace(0, 200, 5000).repeat(4, 1)
    z[1] *= 0.3
    z[2, 1:] -= 30
    z[3, ::2] = -math.inf
    for how in (dict(top_k=4000), dict(top_k=2, top_p=0.5), dict(top_k=3000, top_p=0.9), dict(top_p=0.9999)):
        check(dev, z, uniforms(4, 12), **how)


def test_rows_without_a_distribution():
    dev = cuda_or_skip()
    z = logits(9, 700, 13)
    z[1, 699] = math.nan
    z[2, 0] = math.inf
    z[3] = -math.inf
    tau = torch.ones(9)
    tau[4], tau[5], tau[6] = math.nan, -1.0, math.inf
    p = torch.full((9,), 0.9)
    p[7] = math.nan
    for how in (dict(), dict(top_k=5)):
        token, logp = check(dev, z, uniforms(9, 14), temperature=tau, top_p=p, **how)
        assert (token[1:8] == -1).all() and token[0] >= 0 and token[8] >= 0
    u = uniforms(9, 14)
    u[0] = math.nan
    token, _ = rlk.sample_logits(z.to(dev), u.to(dev))
    assert token[0] == -1 and token[8] >= 0


def test_uniform_numbers_at_their_ends():
    dev = cuda_or_skip()
    z = logits(6, 900, 15)
    z[:, 899] = -math.inf
    u = torch.tensor([0.0, 1.0 - 2.0 ** -53, 1.0, -0.5, 2.0 ** -31, 1.0 - 2.0 ** -31], dtype=torch.float64)
    token, _ = check(dev, z, u)
    assert token[0] == 0 and (token[1:3] == 898).all() and token[3] == 0
    check(dev, z, u.float().clamp(max=1 - 2.0 ** -24), top_p=0.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layouts(dtype):
    """Odd pitches, starts at every place of a 16-byte vector, leading dims, strided settings and
    uniforms: the same tokens and bits."""
    dev = cuda_or_skip()
    N, V = 12, 2051
    z = logits(N, V, 16).to(dtype).to(dev)
    u = uniforms(N, 17).to(dev)
    how = dict(temperature=0.8, top_k=40, top_p=0.9)
    want = check(dev, z, u.cpu(), **how)
    for shift in range(9):
        wide = torch.full((N, V + 13), 99.0, dtype=dtype, device=dev)   # neighbours must not matter
        wide[:, shift:shift + V] = z
        for settings in (how, dict()):
            a = rlk.sample_logits(wide[:, shift:shift + V], u, **settings)
            b = want if settings else rlk.sample_logits(z, u)
            assert torch.equal(a[0], b[0]) and bits_equal(a[1], b[1])
    token, logp = rlk.sample_logits(z.view(3, 4, V), u.view(3, 4), **how)
    assert token.shape == (3, 4) and torch.equal(token.view(-1), want[0])
    pair = torch.stack([u, u], 1)
    tau = torch.full((N, 2), 0.8, device=dev)
    a = rlk.sample_logits(z.t().contiguous().t(), pair[:, 1], temperature=tau[:, 0], top_k=40, top_p=0.9)
    assert torch.equal(a[0], want[0]) and bits_equal(a[1], want[1])


def test_rows_do_not_depend_on_the_call():
    """One row, some rows, all rows (other cluster sizes), another order, another stream, repeats,
    and a replayed graph."""
    dev = cuda_or_skip()
    N, V = 300, 9001
    z, u = logits(N, V, 18).to(dev), uniforms(N, 19).to(dev)
    for how in (dict(), dict(top_p=0.9), dict(top_k=60, top_p=0.9, temperature=0.9)):
        token, logp = rlk.sample_logits(z, u, **how)
        for s in (slice(0, 1), slice(17, 18), slice(5, 25), slice(100, 239)):
            a = rlk.sample_logits(z[s], u[s], **how)
            assert torch.equal(a[0], token[s]) and bits_equal(a[1], logp[s])
        back = torch.arange(N - 1, -1, -1, device=dev)
        a = rlk.sample_logits(z[back], u[back], **how)
        assert torch.equal(a[0][back], token) and bits_equal(a[1][back], logp)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        a = rlk.sample_logits(z, u, stream=side, **how)
        side.synchronize()
        assert torch.equal(a[0], token) and bits_equal(a[1], logp)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a = rlk.sample_logits(z, u, **how)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a[0], token) and bits_equal(a[1], logp)


def test_many_rows_on_a_stream_and_in_a_graph():
    dev = cuda_or_skip()
    z, u = kinds(120, 20000, 24).to(dev), uniforms(120, 25).to(dev)
    for how in (dict(top_p=0.9), dict(top_k=60, top_p=0.9), dict(top_k=2000)):
        token, logp = rlk.sample_logits(z, u, **how)
        for _ in range(3):
            a = rlk.sample_logits(z, u, **how)
            assert torch.equal(a[0], token) and bits_equal(a[1], logp)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        a = rlk.sample_logits(z, u, stream=side, **how)
        side.synchronize()
        assert torch.equal(a[0], token) and bits_equal(a[1], logp)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a = rlk.sample_logits(z, u, **how)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a[0], token) and bits_equal(a[1], logp)


def test_no_rows_and_refusals():
    dev = cuda_or_skip()
    z, u = logits(4, 100, 20).to(dev), uniforms(4, 21).to(dev)
    token, logp = rlk.sample_logits(z[:0], u[:0], top_k=3)
    assert token.shape == (0,) and logp.shape == (0,) and token.dtype == torch.int64
    for bad in (dict(temperature=-1.0), dict(temperature=math.nan), dict(temperature=math.inf),
                dict(top_p=math.nan), dict(min_p=math.nan)):
        with pytest.raises(rlk.RlkError, match="RLK_ERR_VALUE"):
            rlk.sample_logits(z, u, **bad)
    for bad, error in ((dict(temperature=torch.ones(3, device=dev)), ValueError),
                       (dict(top_k=torch.ones(4, device=dev)), TypeError),
                       (dict(top_p=torch.ones(4)), ValueError)):
        with pytest.raises(error):
            rlk.sample_logits(z, u, **bad)
    with pytest.raises(TypeError):
        rlk.sample_logits(z.double(), u)
    with pytest.raises(ValueError):
        rlk.sample_logits(z, u[:3])
