"""The selective scan's step sizes: a bias of its own without softplus, states that grow, channels that do not fill a
wavefront; every gradient, forwards, backwards and token by token, with the tolerances of test_sel_scan.py (a step size off by
at most 8 roundings: here the sum with the bias alone).  Growing states' A is positive throughout, so that the
magnitudes' two parts of a step size have one sign; a decay above one is off by as many roundings of |delta A| as one below."""
import pytest
import torch

import chunked_gated_delta_12_amd as kda
from test_sel_scan import BF16, DEV, F32, check_bwd, check_fwd, cu_of, inputs, options, spans, to_dev

pytestmark = pytest.mark.gpu


def steps(x, bias, least, most, seed):
    """dt = -bias + a step within [least, most], as it is stored; fp32 keeps the sum's step exact to a rounding, bf16 to 2^-8 of dt,
    which at a bias of 1 stays above zero for steps from 2^-6 on."""
    gen = torch.Generator().manual_seed(seed)
    D = x["A"].shape[0]
    x["dt_bias"] = torch.full((D,), float(bias))
    size = least + (most - least) * torch.rand(x["dt"].shape, generator=gen)
    x["dt"] = (size - bias).to(x["dt"].dtype)
    assert (x["dt"].double() + x["dt_bias"].double() > 0).all()
    return x


def both(x, lens, dtype, last=True):
    B, rows, D = x["x"].shape
    N, n = x["A"].shape[1], len(lens) if lens else B
    gen = torch.Generator().manual_seed(8)
    dy = torch.randn(B, rows, D, generator=gen).to(dtype)
    dS = 0.3 * torch.randn(n, D, N, generator=gen) if last else None
    d, cu, sp = to_dev(x), cu_of(lens) if lens else None, spans(B, rows, lens)
    args = (d["x"], d["dt"], d["A"], d["b"], d["c"])
    y, S_T = kda.kda_sel_scan_fwd(*args, d["S0"], cu_seqlens=cu, **options(d, False))
    torch.cuda.synchronize()
    check_fwd(x, y.cpu(), S_T.cpu(), sp, False, dtype)
    got = kda.kda_sel_scan_bwd(*args, dy.to(DEV), d["S0"], None if dS is None else dS.to(DEV), cu_seqlens=cu, **options(d, False))
    torch.cuda.synchronize()
    check_bwd(got, x, dy, dS, sp, False, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,D,N,G", [(1, 33, 32, 16, 1), (2, 150, 72, 8, 1), (1, [5, 0, 1, 64, 65, 0], 48, 16, 2), (1, [200, 1, 129], 24, 32, 1), (1, 40, 136, 64, 1)])
def test_bias_without_softplus(B, T, D, N, G, dtype):
    """Small steps out of a dt and a bias of opposite sign: what has no channel or token reads a dt of zero, and a step of the
    bias alone would be e^16 a token there."""
    print(f"scan B={B} T={T} D={D} N={N} G={G} {dtype}", flush=True)
    lens, rows = (T, sum(T)) if isinstance(T, list) else (None, T)
    x = inputs(B, rows, D, N, G, dtype, 5, "skip z S0", False, len(lens) if lens else None)
    both(steps(x, -1.0, 2.0 ** -5, 2.0 ** -4, 6), lens, dtype)


@pytest.mark.parametrize("bias", [None, 1.0])
@pytest.mark.parametrize("B,T,D,N", [(1, 70, 24, 16), (2, 200, 72, 16), (1, [130, 3, 100], 40, 8)])
def test_growing_states(B, T, D, N, bias):
    """A above zero: a state grows by up to e^(0.3 * 0.06 * 200) = 37."""
    print(f"scan growing B={B} T={T} D={D} N={N} bias={bias}", flush=True)
    lens, rows = (T, sum(T)) if isinstance(T, list) else (None, T)
    x = inputs(B, rows, D, N, 1, F32, 7, "skip z S0", False, len(lens) if lens else None)
    x["A"] = 0.3 * torch.rand(D, N, generator=torch.Generator().manual_seed(3)) + 1e-3
    x = steps(x, bias or 0.0, 2.0 ** -7, 0.06, 4)
    if bias is None:
        x["dt_bias"] = None
    both(x, lens, F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,D,N,G", [(3, 1, 24, 16, 1), (2, 7, 72, 8, 1), (2, 5, 48, 32, 2)])
def test_step_bias_without_softplus(B, T, D, N, G, dtype):
    x = steps(inputs(B, T, D, N, G, dtype, 5, "skip z S0", False), -1.0, 2.0 ** -5, 2.0 ** -4, 6)
    d = to_dev(x)
    y = kda.kda_sel_scan_step(d["x"], d["dt"], d["A"], d["b"], d["c"], d["S0"], **options(d, False))
    torch.cuda.synchronize()
    check_fwd(x, y.cpu(), d["S0"].cpu(), spans(B, T, None), False, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("softplus,A,bias", [(False, -16.0, -1.0), (True, 2.0, 4.0)])
def test_channels_beside_the_group(softplus, A, bias, dtype):
    """Lanes beyond a group's last channel add nothing to db and dc, whatever a step of the bias alone would make of their states:
    a bias alone is e^16 or e^8 a token, its channels' own steps are e^-0.5 and e^0.014."""
    B, T, D, N = 1, 150, 32, 16
    x = inputs(B, T, D, N, 1, dtype, 5, "S0", softplus)
    x["A"] = torch.full((D, N), A)
    x["dt_bias"] = torch.full((D,), bias)
    x["dt"] = torch.full((B, T, D), -9.0 if softplus else 1.0 + 2.0 ** -5).to(dtype)
    d, dy = to_dev(x), torch.ones(B, T, D, dtype=dtype, device=DEV)
    got = kda.kda_sel_scan_bwd(d["x"], d["dt"], d["A"], d["b"], d["c"], dy, d["S0"], torch.ones(B, D, N, device=DEV), **options(d, softplus))
    torch.cuda.synchronize()
    for k in ("dx", "ddt", "dA", "db", "dc", "ddt_bias", "dS0"):
        assert torch.isfinite(got[k]).all(), k
    check_bwd({k: None if v is None else v.cpu() for k, v in got.items()}, x, dy.cpu(), torch.ones(B, D, N), [(0, 0, T)], softplus, dtype)
