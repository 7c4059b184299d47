"""Calls of the state-space operators that stand beside the ordinary ones: captured packed calls whose offsets change
between replays, gradients beside values that are not finite, pools that hundreds of rows name several times."""
import pytest
import torch

import chunked_gated_delta_12_amd as kda
from test_sel_scan import BF16, DEV, F32, NAMES, cu_of, gradients64, inputs, options, spans, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,N", [(2048, 8), (72, 16)])
def test_captured_packed_calls_take_other_offsets(D, N):
    """The lengths are read when the work runs: a graph replayed with other offsets in the same tensor equals the eager calls with
    them bit for bit, whether sequences are cut, empty, or leave rows to none."""
    rows, n = 400, 100
    gen = torch.Generator().manual_seed(3)
    offsets = []
    for most in (rows, 390, 2 * rows, 300):
        cuts = torch.sort(torch.randint(0, most, (n + 1,), generator=gen).clamp_max(rows)).values
        cuts[50:] = torch.clamp_min(cuts[50:], int(cuts[49]) + 150).clamp_max(rows)   # one of 150 tokens and more
        offsets.append(cuts.to(torch.int32).to(DEV))
    x = to_dev(inputs(1, rows, D, N, 1, BF16, 2, "skip z dt_bias S0", True, n))
    w, taps = torch.randn(D, 4, generator=gen).to(DEV), torch.randn(n, 3, D, generator=gen).to(BF16).to(DEV)
    dy, dS = torch.randn(1, rows, D, generator=gen).to(BF16).to(DEV), torch.randn(n, D, N, generator=gen).to(DEV)
    cu = offsets[0].clone()

    def call(cu):
        args = (x["x"], x["dt"], x["A"], x["b"], x["c"])
        y, S = kda.kda_sel_scan_fwd(*args, x["S0"], cu_seqlens=cu, **options(x, True))
        g = kda.kda_sel_scan_bwd(*args, dy, x["S0"], dS, cu_seqlens=cu, **options(x, True))
        yc, Sc = kda.kda_short_conv_fwd(x["x"], w, taps, act="silu", cu_seqlens=cu)
        gc = kda.kda_short_conv_bwd(x["x"], w, dy, taps, taps, act="silu", cu_seqlens=cu)
        return [y, S, yc, Sc] + [g[k] for k in NAMES] + [gc[k] for k in ("dx", "dw", "dS0")]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(cu)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(cu)
    for i in (1, 0, 2, 3, 1):
        cu.copy_(offsets[i])
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(out, call(offsets[i]))):
            assert torch.equal(a, b), (i, k)


@pytest.mark.parametrize("T", [70, 300])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_beside_values_that_are_not_finite(T, dtype):
    """A gradient is finite wherever the definition's is: NaN in one channel's x or dy reaches that channel and its group's db and dc
    where they take it, other channels, groups and sequences are as without it; 24 channels a group leave lanes without one."""
    B, D, N, G = 4, 48, 16, 2
    x = inputs(B, T, D, N, G, dtype, 7, "skip z dt_bias S0")
    gen = torch.Generator().manual_seed(2)
    dy, dS = torch.randn(B, T, D, generator=gen).to(dtype), torch.randn(B, D, N, generator=gen)
    clean = kda_bwd(x, dy, dS)
    x["x"][0, 20, 23] = float("nan")
    dy[1, 30, 47] = float("nan")
    x["S0"][2, 5, 3] = float("inf")
    got = kda_bwd(x, dy, dS)
    want = gradients64(x, dy, dS, spans(B, T, None), True)[0]
    for k in NAMES:
        fine = torch.isfinite(want[k])
        assert torch.isfinite(got[k])[fine].all(), k
        assert fine.any() and not fine.all() or k == "dS0", k
        if k in ("dx", "ddt", "dz", "db", "dc", "dS0"):
            assert torch.equal(got[k][3], clean[k][3]), k


def kda_bwd(x, dy, dS):
    d = to_dev(x)
    g = kda.kda_sel_scan_bwd(d["x"], d["dt"], d["A"], d["b"], d["c"], dy.to(DEV), d["S0"], dS.to(DEV), **options(d, True))
    torch.cuda.synchronize()
    return {k: v.cpu() for k, v in g.items()}


def test_pools_named_many_times():
    """700 rows, 40 slots: the first row with tokens has its slot, the others are padding, at any distance."""
    B, T, D, N, P = 700, 2, 8, 8, 40
    gen = torch.Generator().manual_seed(4)
    slots = torch.randint(-3, P + 3, (B,), generator=gen)
    slots[600:640] = torch.arange(P)
    ntok = torch.randint(0, T + 1, (B,), generator=gen)
    ntok[:300] *= (torch.rand(300, generator=gen) < 0.03).long()
    first = {}
    for i in range(B):
        s = int(slots[i])
        if 0 <= s < P and ntok[i] > 0:
            first.setdefault(s, i)
    assert len(first) == P and max(first.values()) > 256
    rows = torch.tensor([first[s] for s in range(P)])
    x = inputs(B, T, D, N, 1, F32, 6, "skip z dt_bias S0", True, P)
    w, taps = torch.randn(D, 4, generator=gen).to(DEV), torch.randn(P, 3, D, generator=gen)
    d = to_dev(x)
    i32 = lambda t: t.to(torch.int32).to(DEV)   # noqa: E731

    def both(at, slots, ntok):
        S, C, y0 = d["S0"].clone(), taps.to(DEV), torch.full((len(at), T, D), 7.0, device=DEV)
        e = {k: d[k][at].contiguous() for k in ("x", "dt", "b", "c", "z")}
        y = kda.kda_sel_scan_step(e["x"], e["dt"], d["A"], e["b"], e["c"], S, slots=slots, ntok=i32(ntok), y=y0.clone(),
                                  skip=d["skip"], z=e["z"], dt_bias=d["dt_bias"])
        c = kda.kda_short_conv_step(e["x"], w, C, act="silu", slots=slots, ntok=i32(ntok), y=y0.clone())
        return [t.cpu() for t in (y, c)], [t.cpu() for t in (S, C)]

    y, S = both(torch.arange(B), i32(slots), ntok)
    one_y, one_S = both(rows, None, ntok[rows])   # each slot's row alone
    others = torch.ones(B, dtype=torch.bool)
    others[rows] = False
    for a, b in zip(S, one_S):
        assert torch.equal(a, b)
    for a, b in zip(y, one_y):
        assert torch.equal(a[rows], b)
        assert (a[others] == 7).all()
