"""The selective scan over sequences of many pieces, where the joins of the pieces' maps carry what is compared: inputs in
the first 40 tokens alone and gradients of the last 40 alone, with decays of e^-2.6 at most over the whole, so that every
value at the other end went through every piece.  64 tokens a piece: up to 8, 4 and 2 pieces are joined at a time (16, 32 and 64
states), so these have full batches, part batches and several of them in both directions.  Tolerances are test_sel_scan.py's, and
are far below what is carried (checked on the CPU)."""
import pytest
import torch

import chunked_gated_delta_12_amd as kda
from plain_ops import U32
from test_sel_scan import BF16, DEV, F32, check_bwd, check_fwd, cu_of, gradients64, inputs, options, spans, to_dev

FAR = 40


def far(B, rows, D, N, dtype, sp, seed=31):
    x = inputs(B, rows, D, N, 1, dtype, seed, "skip z dt_bias S0", True, len(sp))
    gen = torch.Generator().manual_seed(seed + 1)
    x["A"] = -(0.02 + 0.18 * torch.rand(D, N, generator=gen))
    x["dt_bias"] = torch.full((D,), -4.0)   # steps of 0.018
    x["dt"] = (0.1 * torch.randn(B, rows, D, generator=gen)).to(dtype)
    dy, dS = torch.randn(B, rows, D, generator=gen).to(dtype), 0.3 * torch.randn(len(sp), D, N, generator=gen)
    for i, lo, hi in sp:
        x["x"][i, lo + FAR:hi] = 0
        dy[i, lo:max(lo, hi - FAR)] = 0
    return x, dy, dS


CASES = [  # B, T or lengths, D, N
    (1, 700, 64, 16), (2, 600, 24, 16), (1, 1100, 8, 8), (1, 420, 64, 64), (1, 700, 32, 32), (1, [90, 700, 0, 65, 530], 72, 16)]


def case(B, T, D, N, dtype):
    lens, rows = (T, sum(T)) if isinstance(T, list) else (None, T)
    sp = spans(B, rows, lens)
    return lens, rows, sp, far(B, rows, D, N, dtype, sp)


@pytest.mark.parametrize("B,T,D,N", CASES)
def test_what_is_carried_shows(B, T, D, N):
    lens, rows, sp, (x, dy, dS) = case(B, T, D, N, F32)
    g, mag, r = gradients64(x, dy, dS, sp, True)
    assert r * U32 < 2e-3
    n, (i, lo, hi) = max(enumerate(sp), key=lambda s: s[1][2] - s[1][1])
    for k, at in (("dx", slice(lo, lo + FAR)), ("db", slice(lo, lo + FAR)), ("dc", slice(hi - FAR, hi)), ("dz", slice(hi - FAR, hi))):
        v, tol = g[k][i, at].abs(), r * U32 * mag[k][i, at]
        assert (v > 10 * tol).double().mean() > 0.8, k
    assert (g["dS0"][n].abs() > 10 * r * U32 * mag["dS0"][n]).double().mean() > 0.8


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,D,N", CASES)
def test_joins(B, T, D, N, dtype):
    print(f"scan joins B={B} T={T} D={D} N={N} {dtype}", flush=True)
    lens, rows, sp, (x, dy, dS) = case(B, T, D, N, dtype)
    d, cu = to_dev(x), cu_of(lens) if lens else None
    args = (d["x"], d["dt"], d["A"], d["b"], d["c"])
    y, S_T = kda.kda_sel_scan_fwd(*args, d["S0"], cu_seqlens=cu, **options(d, True))
    got = kda.kda_sel_scan_bwd(*args, dy.to(DEV), d["S0"], dS.to(DEV), cu_seqlens=cu, **options(d, True))
    torch.cuda.synchronize()
    check_fwd(x, y.cpu(), S_T.cpu(), sp, True, dtype)
    check_bwd(got, x, dy, dS, sp, True, dtype)
