"""Tensors of more than 2^31 elements through the operators of a state-space block: what the last tokens
give in one call over all rows equals a call over these tokens alone, from the state that the rows before them
leave.  The states of both come from the same kernels, so they differ by less than 2^-16 (test_sel_scan.py's
bound at the step sizes here, a few roundings a token over the thousand tokens that a state remembers), and results
in bf16 by one step, 2^-7 of them, where that falls next to a border."""
import pytest
import torch

import chunked_gated_delta_12_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T, D, N, LAST = (1 << 19) + 77, 4096, 8, 40


@pytest.fixture(scope="module")
def x():
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(1, T, D, generator=gen, device=DEV, dtype=torch.bfloat16)
    assert x.numel() > 1 << 31
    yield x
    torch.cuda.empty_cache()


def near(got, want, what):
    print(what, flush=True)
    a, b = got.double(), want.double()
    tol = 2.0 ** -7 * b.abs() + 2.0 ** -16 * b.abs().max()
    assert ((a - b).abs() <= tol).all(), f"{what}: {(a - b).abs().max().item():.3g}"


def test_short_conv(x):
    w = torch.randn(D, 4, generator=torch.Generator().manual_seed(2)).to(DEV)
    y, S = kda.kda_short_conv_fwd(x, w, act="silu")
    _, before = kda.kda_short_conv_fwd(x[:, :-LAST], w, act="silu")
    tail = x[:, -LAST:].contiguous()
    near(y[:, -LAST:], kda.kda_short_conv_fwd(tail, w, before, act="silu")[0], "y")
    assert torch.equal(S[0], x[0, -3:])
    del y
    g = kda.kda_short_conv_bwd(x, w, x, act="silu", want_dS0=False)["dx"]
    near(g[:, -LAST:], kda.kda_short_conv_bwd(tail, w, tail, before, act="silu")["dx"], "dx")


def test_layer_norm(x):
    _, h = kda.kda_layer_norm_fwd(x)
    tail = x[:, -LAST:].contiguous()
    near(h[:, -LAST:], kda.kda_layer_norm_fwd(tail)[1], "h")
    d = kda.kda_layer_norm_bwd(x, x, want_db=False)["dy"]
    near(d[:, -LAST:], kda.kda_layer_norm_bwd(tail, tail, want_db=False)["dy"], "dy")


def test_sel_scan(x):
    gen = torch.Generator(device=DEV).manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)   # noqa: E731
    b, c = (r(1, T, 1, N).to(torch.bfloat16) for _ in range(2))
    A, bias = -torch.exp(r(D, N)), torch.full((D,), -5.0, device=DEV)
    tail, tb, tc = (t[:, -LAST:].contiguous() for t in (x, b, c))
    y, S = kda.kda_sel_scan_fwd(x, x, A, b, c, dt_bias=bias)
    _, before = kda.kda_sel_scan_fwd(x[:, :-LAST], x[:, :-LAST], A, b[:, :-LAST], c[:, :-LAST], dt_bias=bias)
    want, want_S = kda.kda_sel_scan_fwd(tail, tail, A, tb, tc, before, dt_bias=bias)
    near(y[:, -LAST:], want, "y")
    near(S, want_S, "S_T")
    del y
    g = kda.kda_sel_scan_bwd(x, x, A, b, c, x, dt_bias=bias, want_dS0=False)
    w = kda.kda_sel_scan_bwd(tail, tail, A, tb, tc, tail, before, dt_bias=bias)
    for k in ("dx", "ddt", "db", "dc"):
        near(g[k][:, -LAST:], w[k], k)
