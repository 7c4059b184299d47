"""Results of the selective scan that are fp32 whatever the storage (states, weights' gradients) have fp32 precision in both.

One token with x, b, c and dy of 1 and no start state, so that products and sums around a value are exact: the last state
is the step size softplus(v), ddt_bias is N slopes of it, and dskip the gate silu(z).  In roundings of 2^-24 of the
value: e^-|v| has 2 for the hardware's exponential, 1 for the correction's product and, from ln 2's own rounding,
0.046 |v|; softplus adds 1 for 2 + e, 2 for a reciprocal, 1 for a product, 2 for the series and its sum, and 1 more; the
slope and the gate fewer.  So they are off by at most 12 + 0.05 |v|.  (An exponential of a rounded -|v| log2(e) alone is off by up to
22 + 0.22 |v| from |v| = 22 on, 11 + 0.22 |v| from 11 on.)
"""
import math

import pytest
import torch

import chunked_gated_delta_12_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
D, N = 4096, 8


def near(got, want, v, what):
    got, v = got.double().cpu(), v.double()
    tol = (12 + 0.05 * v.abs()) * 2.0 ** -24 * want
    bad = (got - want).abs() > tol
    i = torch.argmax((got - want).abs() / tol).item()
    assert not bad.any(), f"{what}: {int(bad.sum())} of {D} off; at {v[i].item():.6g} by {((got[i] - want[i]) / want[i]).item() * 2 ** 24:.1f} roundings"


def ones(dtype):
    one = lambda *s: torch.ones(*s, dtype=dtype, device=DEV)   # noqa: E731
    return dict(x=one(1, 1, D), b=one(1, 1, 1, N), c=one(1, 1, 1, N), A=-torch.ones(D, N, device=DEV))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_step_sizes(dtype):
    a = ones(dtype)
    v = torch.linspace(-80, 20, D)
    bias, dt = v.to(DEV), torch.zeros(1, 1, D, dtype=dtype, device=DEV)
    v64 = v.double()
    delta = torch.where(v64 > 0, v64, 0.0) + torch.log1p(torch.exp(-v64.abs()))
    _, S = kda.kda_sel_scan_fwd(a["x"], dt, a["A"], a["b"], a["c"], dt_bias=bias)
    pool = torch.zeros(1, D, N, device=DEV)
    kda.kda_sel_scan_step(a["x"], dt, a["A"], a["b"], a["c"], pool, dt_bias=bias)
    for state, what in ((S, "S_T"), (pool, "the pool's state")):
        assert (state == state[..., :1]).all()
        near(state[0, :, 0], delta, v, what)
    g = kda.kda_sel_scan_bwd(a["x"], dt, a["A"], a["b"], a["c"], a["x"], dt_bias=bias)
    near(g["ddt_bias"], N * torch.sigmoid(v64), v, "ddt_bias")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gates(dtype):
    a = ones(dtype)
    z = torch.linspace(-60, 20, D).to(dtype)
    dt = torch.zeros(1, 1, D, dtype=dtype, device=DEV)
    g = kda.kda_sel_scan_bwd(a["x"], dt, a["A"], a["b"], a["c"], a["x"], z=z.view(1, 1, D).to(DEV), skip=torch.ones(D, device=DEV))
    z64 = z.double()
    near(g["dskip"] * torch.sign(z).to(DEV), (z64 * torch.sigmoid(z64)).abs(), z, "dskip")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("low", ["lowest", "-inf"])
def test_masked_steps(low, dtype):
    """A dt of the type's lowest value or of minus infinity is a step of nothing: the state is kept bit for bit, the token's
    gradients are zero or its skip's."""
    T, n = 40, 64
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen).to(DEV)   # noqa: E731
    dt = torch.full((1, T, n), torch.finfo(dtype).min if low == "lowest" else -math.inf, dtype=dtype, device=DEV)
    x, dy, z, b, c = (r(*s).to(dtype) for s in ((1, T, n), (1, T, n), (1, T, n), (1, T, 1, N), (1, T, 1, N)))
    A, S0, dS, skip, bias = -r(n, N).abs(), r(1, n, N), r(1, n, N), r(n), r(n)
    opt = dict(skip=skip, z=z, dt_bias=bias)
    y, S = kda.kda_sel_scan_fwd(x, dt, A, b, c, S0, **opt)
    assert torch.equal(S, S0) and torch.isfinite(y).all()
    pool = S0.clone()
    kda.kda_sel_scan_step(x, dt, A, b, c, pool, **opt)
    assert torch.equal(pool, S0)
    g = kda.kda_sel_scan_bwd(x, dt, A, b, c, dy, S0, dS, **opt)
    assert all(torch.isfinite(v).all() for v in g.values())
    assert not g["ddt"].any() and not g["dA"].any() and not g["db"].any() and not g["ddt_bias"].any()
    gate = z.double() * torch.sigmoid(z.double())
    want = skip.double() * dy.double() * gate
    assert ((g["dx"].double() - want).abs() <= 2.0 ** -7 * want.abs() + 1e-30).all()
