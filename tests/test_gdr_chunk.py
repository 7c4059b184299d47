"""kda_gdr_chunk_fwd and kda_gdr_chunk_bwd against the token-by-token definition in 64 bits
(gradients by autograd through it).

Tolerances, as a share of the largest value of a result.  With unit keys, 0 <= beta <= 1 and
g <= 0 a token's map of the state has norm at most one, so errors of earlier chunks do not
grow and what a chunk adds counts.  bf16 storage: an operand split in two bf16 halves is off
by at most 2^-18 of itself and the halves' product that is left out is 2^-18, so a product
adds at most 3 * 2^-18 < 2^-16 of the terms it sums; a chunk runs through eight such products
one behind another (state, X, U, state; P, output), whose terms sum to no more than a few times the
results here: 8 * 2^-16 * 2 = 2^-12.  fp32 storage: the same eight, each a sum of at most 128
products with one rounding of 2^-24 a term: 8 * 128 * 2^-24 = 2^-14; an exponential of
|g| <= 120 adds 120 roundings, which is less.  Gradients run through both chains: twice
that.  Values stored in bf16 are rounded once more, by at most 2^-8 of themselves.
"""
import ctypes

import pytest
import torch

import chunked_gated_delta_12_amd as kda
from plain_ops import HALF_STEP, gdr_inputs, gdr_tokens

DEV = "cuda:0"
FWD = {torch.bfloat16: 2.0 ** -12, torch.float32: 2.0 ** -14}


def near(got, ref, dtype, share, what):
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, what
    assert got.isfinite().all(), what
    top = float(ref.abs().max()) if ref.numel() else 0.0
    tol = share * top + HALF_STEP[dtype] * (ref.abs() + share * top) + 1e-37
    err = (got - ref).abs()
    if not (err <= tol).all():
        i = int((err / tol).argmax())
        raise AssertionError(f"{what}: {int((err > tol).sum())} of {err.numel()} off; worst at {i}: got "
                             f"{got.reshape(-1)[i]:.8g}, want {ref.reshape(-1)[i]:.8g}, top {top:.4g}")


def offsets(lens, head=0):
    cu = [head]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def make(lens, Hk, Hv, dk, dv, dtype, seed, head=0, tail=0, s0=True, **kw):
    cu = offsets(lens, head)
    x = gdr_inputs((1, cu[-1] + tail), Hk, Hv, dk, dv, dtype, seed, **kw)
    gen = torch.Generator().manual_seed(seed + 1)
    n = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    x["S0"] = 0.2 * n(len(lens), Hv, dk, dv) if s0 else None
    x["do"] = n(1, cu[-1] + tail, Hv, dv).to(dtype)
    x["dS_T"] = 0.2 * n(len(lens), Hv, dk, dv) if s0 else None
    return x, cu


def to(x, dev=DEV):
    return {k: None if v is None else v.to(dev) for k, v in x.items()}


def reference(x, cu, scale, grads):
    """o, S_T and, asked for, the gradients, each over all rows (zero for rows of no sequence)."""
    leaf = {k: x[k].double().requires_grad_(grads) for k in ("q", "k", "v", "g", "beta")}
    N, Hv, dk, dv = len(cu) - 1, x["v"].shape[2], x["q"].shape[3], x["v"].shape[3]
    S0 = torch.zeros(N, Hv, dk, dv, dtype=torch.float64) if x["S0"] is None else x["S0"].double()
    S0 = S0.requires_grad_(grads)
    o = torch.zeros(x["v"].shape, dtype=torch.float64)
    parts, last = [], []
    for i in range(N):
        a = slice(cu[i], cu[i + 1])
        oi, Si = gdr_tokens(*(leaf[k][0, a] for k in ("q", "k", "v", "g", "beta")), S0[i], scale)
        parts.append((a, oi))
        last.append(Si)
        o[0, a] = oi.detach()
    S_T = torch.stack(last)
    if not grads:
        return o, S_T.detach(), None
    loss = sum((oi * x["do"][0, a].double()).sum() for a, oi in parts)
    if x["dS_T"] is not None:
        loss = loss + (S_T * x["dS_T"].double()).sum()
    got = torch.autograd.grad(loss, [leaf[k] for k in ("q", "k", "v", "g", "beta")] + [S0],
                              materialize_grads=True)   # a sequence of no tokens uses none
    return o, S_T.detach(), dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dS0"), got))


def run_fwd(x, cu, scale, **kw):
    d = to(x)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    o, S_T = kda.kda_gdr_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["S0"], cu_seqlens=c, scale=scale, **kw)
    torch.cuda.synchronize()
    return o, S_T


def run_bwd(x, cu, scale, **kw):
    d = to(x)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    r = kda.kda_gdr_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"], d["S0"], d["dS_T"], cu_seqlens=c, scale=scale, **kw)
    torch.cuda.synchronize()
    return r


def check(x, cu, scale, dtype, bwd=True):
    lens = [b - a for a, b in zip(cu, cu[1:])]
    print(f"gdr lens={lens} q={tuple(x['q'].shape)} v={tuple(x['v'].shape)} {dtype}", flush=True)
    o64, S64, g64 = reference(x, cu, scale, bwd)
    o, S_T = run_fwd(x, cu, scale)
    near(o, o64, dtype, FWD[dtype], "o")
    near(S_T, S64, torch.float32, FWD[dtype], "S_T")
    if bwd:
        g = run_bwd(x, cu, scale)
        for k in ("dq", "dk", "dv"):
            near(g[k], g64[k], dtype, 2 * FWD[dtype], k)
        for k in ("dg", "dbeta", "dS0"):
            near(g[k], g64[k], torch.float32, 2 * FWD[dtype], k)


SHAPES = [(1, 1, 32, 32), (2, 4, 64, 64), (1, 3, 128, 128), (2, 2, 64, 96), (1, 2, 128, 256), (1, 4, 32, 160)]
both = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])


@pytest.mark.gpu
@both
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 63, 64, 65, 128, 200])
def test_lengths(T, dtype):
    x, cu = make([T], 1, 2, 64, 64, dtype, T)
    check(x, cu, 0.125, dtype)


@pytest.mark.gpu
@both
@pytest.mark.parametrize("Hk,Hv,dk,dv", SHAPES)
def test_shapes(Hk, Hv, dk, dv, dtype):
    x, cu = make([150], Hk, Hv, dk, dv, dtype, Hv + dk + dv)
    check(x, cu, dk ** -0.5, dtype)


@pytest.mark.gpu
@both
def test_packed(dtype):
    """Sequences of no, one and many tokens, chunks that end inside 64 rows, rows before the
    first and behind the last."""
    x, cu = make([5, 0, 64, 129, 1, 0, 70], 2, 4, 64, 128, dtype, 11, head=3, tail=9)
    check(x, cu, 0.125, dtype)


@pytest.mark.gpu
def test_without_states():
    x, cu = make([130], 1, 1, 128, 64, torch.bfloat16, 12, s0=False)
    check(x, cu, 0.1, torch.bfloat16)
    o, S_T = run_fwd(x, cu, 0.1, want_state=False)
    assert S_T is None
    assert run_bwd(x, cu, 0.1, want_dS0=False)["dS0"] is None


@pytest.mark.gpu
def test_rows_of_no_sequence_are_left_alone():
    x, cu = make([70, 30], 1, 2, 64, 64, torch.bfloat16, 13, head=2, tail=5)
    o = torch.full((1, cu[-1] + 5, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    run_fwd(x, cu, 1.0, o=o)
    assert (o[0, :2] == 7).all() and (o[0, cu[-1]:] == 7).all() and not (o[0, 2:cu[-1]] == 7).all(-1).any()
    g = run_bwd(x, cu, 1.0)
    for k in ("dq", "dk", "dv", "dg", "dbeta"):
        assert not g[k][0, :2].any() and not g[k][0, cu[-1]:].any(), k


@pytest.mark.gpu
@both
def test_dense_equals_packed(dtype):
    x = gdr_inputs((3, 90), 2, 2, 64, 64, dtype, 14)
    d = to(x)
    args = [d[k] for k in ("q", "k", "v", "g", "beta")]
    o, S = kda.kda_gdr_chunk_fwd(*args)
    do = torch.randn(o.shape, generator=torch.Generator().manual_seed(0)).to(dtype).to(DEV)
    gr = kda.kda_gdr_chunk_bwd(*args, do)
    cu = torch.tensor([0, 90, 180, 270], dtype=torch.int32, device=DEV)
    flat = [t.reshape(1, 270, *t.shape[2:]) for t in args]
    o2, S2 = kda.kda_gdr_chunk_fwd(*flat, cu_seqlens=cu)
    gr2 = kda.kda_gdr_chunk_bwd(*flat, do.reshape(1, 270, 2, 64), cu_seqlens=cu)
    assert torch.equal(o.reshape(o2.shape), o2) and torch.equal(S, S2)
    for k in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(gr[k].reshape(gr2[k].shape), gr2[k]), k
    assert torch.equal(gr["dS0"], gr2["dS0"])


@pytest.mark.gpu
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 128), (32, 256)])
def test_many_workgroups(dk, dv):
    """Enough heads that a wavefront takes two column tiles; a few sequences are looked at."""
    lens = [(7 * i) % 140 for i in range(70)]
    x, cu = make(lens, 2, 4, dk, dv, torch.bfloat16, 15)
    o, S_T = run_fwd(x, cu, 0.2)
    g = run_bwd(x, cu, 0.2)
    for i in (1, 9, 20, 69):
        a = slice(cu[i], cu[i + 1])
        y = {k: v[:, a] for k, v in x.items() if k not in ("S0", "dS_T")}
        y["S0"], y["dS_T"] = x["S0"][i:i + 1], x["dS_T"][i:i + 1]
        o64, S64, g64 = reference(y, [0, lens[i]], 0.2, True)
        near(o[:, a], o64, torch.bfloat16, FWD[torch.bfloat16], f"o {i}")
        near(S_T[i:i + 1], S64, torch.float32, FWD[torch.bfloat16], f"S_T {i}")
        for k in ("dq", "dk", "dv", "dg", "dbeta"):
            near(g[k][:, a], g64[k], torch.bfloat16 if k in ("dq", "dk", "dv") else torch.float32, 2 * FWD[torch.bfloat16], f"{k} {i}")
        near(g["dS0"][i:i + 1], g64["dS0"], torch.float32, 2 * FWD[torch.bfloat16], f"dS0 {i}")


@pytest.mark.gpu
@both
@pytest.mark.parametrize("lens,Hk,Hv,dk,dv", [
    ([1500], 1, 2, 64, 64), ([1217], 1, 1, 128, 128), ([30, 1300, 0, 1153, 64], 1, 2, 32, 96), ([1200, 1160], 2, 2, 64, 160)])
def test_cut_sequences(lens, Hk, Hv, dk, dv, dtype):
    """Few heads over long sequences: walked in pieces of a few chunks joined
    by their maps, beside sequences that are not cut."""
    x, cu = make(lens, Hk, Hv, dk, dv, dtype, sum(lens), head=5, tail=2, gmu=-5.0)
    check(x, cu, dk ** -0.5, dtype)


@pytest.mark.gpu
def test_cut_sequence_in_place():
    """The last piece writes S_T while the first has yet to read S0: one buffer for both."""
    x, cu = make([1400], 1, 2, 64, 64, torch.bfloat16, 31, gmu=-6.0)
    o, S = run_fwd(x, cu, 1.0)
    d = to(x)
    for _ in range(3):
        S2 = d["S0"].clone()
        o2, _ = kda.kda_gdr_chunk_fwd(*(d[k] for k in ("q", "k", "v", "g", "beta")), S2, S_T=S2, scale=1.0)
        assert torch.equal(o, o2) and torch.equal(S, S2)


@pytest.mark.gpu
@both
def test_state_in_place_and_resumed(dtype):
    """A sequence in two calls, the second from the first's state written over its start state."""
    x, cu = make([200], 1, 2, 64, 64, dtype, 16)
    o64, S64, _ = reference(x, cu, 0.5, False)
    S = x["S0"].to(DEV)
    outs = []
    for a, b in ((0, 77), (77, 200)):
        y = {k: v[:, a:b].contiguous().to(DEV) for k, v in x.items() if k in ("q", "k", "v", "g", "beta")}
        o, S2 = kda.kda_gdr_chunk_fwd(*(y[k] for k in ("q", "k", "v", "g", "beta")), S, S_T=S, scale=0.5)
        assert S2 is S
        outs.append(o)
    near(torch.cat(outs, 1), o64, dtype, FWD[dtype], "o")
    near(S, S64, torch.float32, FWD[dtype], "S_T")


@pytest.mark.gpu
@both
def test_agrees_with_the_step(dtype):
    x, cu = make([70], 2, 4, 128, 64, dtype, 17)
    o, S_T = run_fwd(x, cu, 0.3)
    d = to(x)
    S = d["S0"].clone()
    o2 = kda.kda_gdr_step(*(d[k] for k in ("q", "k", "v", "g", "beta")), S, scale=0.3)
    near(o, o2.double().cpu(), dtype, FWD[dtype] + 2 * HALF_STEP[dtype], "o")
    near(S_T, S.double().cpu(), torch.float32, FWD[dtype], "S_T")


@pytest.mark.gpu
@both
def test_decays_of_every_size(dtype):
    """Strong decays among weak ones (their sums would take the weak ones' digits), none at
    all, and more than fp32 can hold, forwards and backwards; beta of 0 and 1."""
    x, cu = make([190], 1, 4, 64, 64, dtype, 18, gmu=-6.0)
    x["g"][0, 20, 0], x["g"][0, 70, 0], x["g"][0, 71, 0] = -90.0, -30.0, -1e4
    x["g"][0, :, 1] = 0.0
    x["g"][0, 1::2, 2] = -60.0
    x["beta"][0, 30:60] = 0.0
    x["beta"][0, 90:120] = 1.0
    check(x, cu, 0.125, dtype)


@pytest.mark.gpu
def test_minus_infinity_starts_afresh():
    """g = -inf at a token: what follows is the sequence from there with a state of zero."""
    x, cu = make([150], 1, 2, 64, 64, torch.float32, 19)
    x["g"][0, 83] = float("-inf")
    o, S_T = run_fwd(x, cu, 1.0)
    y = {k: v[:, 83:].contiguous() for k, v in x.items() if k in ("q", "k", "v", "g", "beta")}
    y.update(S0=None, g=y["g"].clone())
    y["g"][0, 0] = 0.0
    o64, S64, _ = reference(y, [0, 67], 1.0, False)
    near(o[:, 83:], o64, torch.float32, FWD[torch.float32], "o")
    near(S_T, S64, torch.float32, FWD[torch.float32], "S_T")
    g = run_bwd(x, cu, 1.0)
    assert all(v.isfinite().all() for v in g.values())
    # and no gradient passes the token: the start state's is that of the tokens before it
    z = {k: v[:, :83].contiguous() for k, v in x.items() if k in ("q", "k", "v", "g", "beta", "do")}
    z.update(S0=x["S0"], dS_T=None)
    near(g["dS0"], reference(z, [0, 83], 1.0, True)[2]["dS0"], torch.float32, 2 * FWD[torch.float32], "dS0")


@pytest.mark.gpu
@both
def test_equal_keys(dtype):
    """One key for all tokens, beta 1: X is as far from the identity as it gets."""
    x, cu = make([100], 1, 1, 64, 64, dtype, 20)
    x["k"][:] = x["k"][:, :1]
    x["beta"][:] = 1.0
    x["g"][:] = -1e-3
    check(x, cu, 0.125, dtype)


@pytest.mark.gpu
def test_nan_stays_in_its_sequence():
    x, cu = make([64, 65, 63], 1, 2, 64, 64, torch.bfloat16, 21)
    o, S_T = run_fwd(x, cu, 1.0)
    g = run_bwd(x, cu, 1.0)
    x["v"][0, 70, 1, 3] = float("nan")
    o2, S2 = run_fwd(x, cu, 1.0)
    g2 = run_bwd(x, cu, 1.0)
    keep = torch.ones(192, dtype=torch.bool)
    keep[64:129] = False
    assert torch.equal(o[0, keep], o2[0, keep]) and torch.equal(S_T[[0, 2]], S2[[0, 2]])
    assert torch.equal(o[0, :, 0], o2[0, :, 0])          # the other head
    assert o2[0, 70, 1, 3].isnan()
    for k in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(g[k][0, keep], g2[k][0, keep]), k


@pytest.mark.gpu
def test_repeats_bit_for_bit_and_on_a_stream():
    x, cu = make([300, 50], 2, 4, 128, 128, torch.bfloat16, 22)
    o, S_T = run_fwd(x, cu, 1.0)
    g = run_bwd(x, cu, 1.0)
    side = torch.cuda.Stream()
    o2, S2 = run_fwd(x, cu, 1.0, stream=side)
    g2 = run_bwd(x, cu, 1.0, stream=side)
    assert torch.equal(o, o2) and torch.equal(S_T, S2)
    for k in g:
        assert torch.equal(g[k], g2[k]), k


@pytest.mark.gpu
def test_captured():
    """Both passes in one graph; lengths and inputs change between replays."""
    x, cu = make([100, 28], 1, 2, 64, 64, torch.bfloat16, 23)
    d = to(x)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    a = [d[k] for k in ("q", "k", "v", "g", "beta")]

    def both_passes():
        o, S = kda.kda_gdr_chunk_fwd(*a, d["S0"], cu_seqlens=c, scale=1.0)
        return [o, S] + [v for _, v in sorted(kda.kda_gdr_chunk_bwd(*a, d["do"], d["S0"], d["dS_T"], cu_seqlens=c, scale=1.0).items())]

    both_passes()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both_passes()
    for i, at in enumerate((100, 3, 64, 128, 0)):
        c.copy_(torch.tensor([0, at, 128], dtype=torch.int32))
        d["v"].copy_(torch.randn(d["v"].shape, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        want = both_passes()
        torch.cuda.synchronize()
        for j, (p, q) in enumerate(zip(got, want)):
            assert torch.equal(p, q), (i, j)


@pytest.mark.gpu
def test_offsets_out_of_order_or_range_touch_nothing_else():
    """The offsets are held to the rows and to their order on the device: the guard rows
    around the tensors keep their values."""
    rows, Hv = 200, 2
    x, _ = make([rows], 1, Hv, 64, 64, torch.bfloat16, 24)
    d = to(x)
    pad = torch.full((rows + 128, Hv, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    o = pad[64:64 + rows].unsqueeze(0)
    for cu in ([0, 150, 100, 200], [-7, 90, 1 << 30, 200], [200, 0, 200, 100], [300, 400, -1, -2]):
        c = torch.tensor(cu, dtype=torch.int32, device=DEV)
        kda.kda_gdr_chunk_fwd(*(d[k] for k in ("q", "k", "v", "g", "beta")), cu_seqlens=c, scale=1.0, o=o)
        torch.cuda.synchronize()
        assert (pad[:64] == 5).all() and (pad[64 + rows:] == 5).all(), cu


@pytest.mark.gpu
def test_rows_past_32_bits():
    """More than 2^31 elements of v and o: the last sequence against the same one alone."""
    Hv, rows, n = 256, 70000, 100
    gen = torch.Generator(device=DEV).manual_seed(0)
    r = lambda *s, dt=torch.bfloat16: torch.randn(*s, generator=gen, device=DEV, dtype=dt)   # noqa: E731
    q, k = (torch.nn.functional.normalize(r(1, rows, 1, 32), dim=-1) for _ in range(2))
    v = r(1, rows, Hv, 128)
    assert v.numel() > 1 << 31
    g, beta = -r(1, rows, Hv, dt=torch.float32).abs(), torch.sigmoid(r(1, rows, Hv, dt=torch.float32))
    cu = torch.tensor([0, rows - n, rows], dtype=torch.int32, device=DEV)
    o, S = kda.kda_gdr_chunk_fwd(q, k, v, g, beta, cu_seqlens=cu, scale=1.0)
    one = [t[:, rows - n:].contiguous() for t in (q, k, v, g, beta)]
    o2, S2 = kda.kda_gdr_chunk_fwd(*one, scale=1.0)
    torch.cuda.synchronize()
    assert torch.equal(o[:, rows - n:], o2) and torch.equal(S[1:], S2)


@pytest.mark.gpu
def test_gradients_by_differences():
    """Central differences of the kernel's own forward in fp32 along one direction an input."""
    x, cu = make([80], 1, 2, 32, 32, torch.float32, 25)
    d = to(x)
    g = run_bwd(x, cu, 1.0)
    names = ("q", "k", "v", "g", "beta", "S0")

    def loss(y):
        o, S = kda.kda_gdr_chunk_fwd(*(y[k] for k in names), scale=1.0)
        return float((o.double() * d["do"].double()).sum() + (S.double() * d["dS_T"].double()).sum())

    gen = torch.Generator().manual_seed(2)
    step = 2.0 ** -7   # truncation of the order 2^-14, roundings 2^-24 * 32 / 2^-7 = 2^-12 of the loss's size
    for k in names:
        u = torch.randn(d[k].shape, generator=gen).to(DEV)
        u = u / u.norm()
        up, down = (loss({**d, k: d[k] + s * step * u}) for s in (1, -1))
        want = float((g["d" + k].double() * u.double()).sum())
        assert abs((up - down) / (2 * step) - want) <= 2.0 ** -8 * float(g["d" + k].double().norm()), k


# ----------------------------------------------------------------------------- refusals (no GPU)
@pytest.fixture(scope="module")
def lib():
    try:
        return kda.load_library()
    except RuntimeError as e:
        pytest.skip(str(e))


FWD_PTRS = ("cu", "q", "k", "v", "g", "beta", "S0", "o", "S_T", "ws")
BWD_PTRS = ("cu", "q", "k", "v", "g", "beta", "S0", "do", "dS_T", "dq", "dk", "dv", "dg", "dbeta", "dS0", "ws")


def caller(fn, order):
    a, base = {}, 1 << 40
    for k in order:
        a[k] = base
        base += 1 << 28

    def call(dtype=0, nseq=2, T=100, Hk=1, Hv=2, dk_=64, dv_=64, scale=1.0, ws_bytes=1 << 28, **over):
        b = {**a, **over}
        return fn(dtype, nseq, T, Hk, Hv, dk_, dv_, scale, *[None if b[k] is None else ctypes.c_void_p(b[k]) for k in order],
                  ws_bytes, None)

    return a, call


@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_refusals(lib, which):
    order = FWD_PTRS if which == "fwd" else BWD_PTRS
    a, call = caller(lib.kda_gdr_chunk_fwd if which == "fwd" else lib.kda_gdr_chunk_bwd, order)
    size = kda.kda_gdr_chunk_fwd_workspace_size if which == "fwd" else kda.kda_gdr_chunk_bwd_workspace_size
    assert call(dtype=2) == 3
    for bad in (dict(nseq=0), dict(T=0), dict(Hk=0), dict(Hk=2, Hv=3), dict(Hv=1, Hk=2), dict(dk_=16), dict(dk_=96), dict(dk_=256),
                dict(dv_=16), dict(dv_=40), dict(dv_=288), dict(scale=float("nan")), dict(scale=float("-inf")),
                dict(nseq=1 << 20, T=1 << 20, cu=None), dict(T=(1 << 31) - 1, Hv=1 << 8, Hk=1)):
        assert call(**bad) == 2, bad
    for k in set(order) - {"cu", "S0", "S_T", "dS_T", "dS0", "ws"}:
        assert call(**{k: None}) == 1, k
    need = size(2, 100, 2, 64, 64, True)
    assert call(ws_bytes=need - 1) == 5 and call(ws=None) == 5
    assert call(cu=None, ws_bytes=size(2, 100, 2, 64, 64, False) - 1) == 5
    assert call(Hk=1 << 18, Hv=1 << 18) == 2            # a chunk's rows past 32-bit offsets
    assert call(q=a["q"] + 8) == 4 and call(cu=a["cu"] + 4) == 4
    if which == "fwd":
        assert call(o=a["v"]) == 6 and call(o=a["S_T"]) == 6 and call(S_T=a["S0"] + 16) == 6 and call(ws=a["cu"]) == 6
    else:
        assert call(dq=a["q"]) == 6 and call(dk=a["dq"]) == 6 and call(dS0=a["dS_T"]) == 6 and call(dv=a["do"]) == 6
        assert call(ws=a["beta"]) == 6


def test_workspace_sizes(lib):
    """Chunks of 64 tokens; packed rows may hold one part chunk a sequence."""
    f = kda.kda_gdr_chunk_fwd_workspace_size
    assert f(3, 64, 2, 64, 64) == f(3, 1, 2, 64, 64) == f(1, 192, 2, 64, 64)
    assert f(3, 65, 2, 64, 64) == 2 * f(3, 64, 2, 64, 64)
    assert f(4, 128, 2, 64, 64, True) == f(6, 64, 2, 64, 64)
    # long sequences of few heads are cut: pieces of 64 chunks here, each with its map and start state
    one = f(1, 64, 1, 128, 128)
    assert f(1, 65536, 16, 128, 128) == 16 * (1024 * one + 16 * (128 * 256 + 128 * 128) * 4)
    assert f(64, 4096, 16, 128, 128) == 64 * 64 * 16 * one
    b = kda.kda_gdr_chunk_bwd_workspace_size
    # X, the tokens' factors, two states and two token operands
    assert b(1, 64, 1, 128, 128) == 6 * 2048 + 4 * 256 + 512 + 2 * 4 * 128 * 128 + 2 * 4 * 64 * 128
    with pytest.raises(kda.KdaError):
        f(0, 64, 2, 64, 64)
    with pytest.raises(kda.KdaError):
        b(1, 64, 2, 64, 48)


def test_binding_refusals(lib):
    x, cu = make([10, 20], 1, 2, 32, 32, torch.float32, 1)
    a = [x[k] for k in ("q", "k", "v", "g", "beta")]
    c = torch.tensor(cu, dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.kda_gdr_chunk_fwd(*a, cu_seqlens=c)                                # not on the GPU
    with pytest.raises(TypeError):
        kda.kda_gdr_chunk_fwd(*a, cu_seqlens=c.long())
    with pytest.raises(ValueError):
        kda.kda_gdr_chunk_fwd(*a, x["S0"][:1], cu_seqlens=c)                   # a state a sequence
    with pytest.raises(ValueError):
        kda.kda_gdr_chunk_fwd(*(t.reshape(2, 15, *t.shape[2:]) for t in a), cu_seqlens=c)
    with pytest.raises(TypeError):
        kda.kda_gdr_chunk_fwd(a[0].half(), *a[1:])
    with pytest.raises(ValueError):
        kda.kda_gdr_chunk_bwd(*a, x["do"][:, :5], cu_seqlens=c)
    with pytest.raises(ValueError):
        kda.kda_gdr_chunk_fwd(a[0], a[1], a[2], a[3][0], a[4], cu_seqlens=c)


@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_workspace_of_the_caller_is_checked(lib, which):
    """What the kernels would write through is refused on the host: another device, a view with gaps, no tensor."""
    x, cu = make([10, 20], 1, 2, 32, 32, torch.float32, 1)
    a = [x[k] for k in ("q", "k", "v", "g", "beta")] + ([x["do"]] if which == "bwd" else [])
    call = kda.kda_gdr_chunk_fwd if which == "fwd" else kda.kda_gdr_chunk_bwd
    with pytest.raises(ValueError, match="workspace is on"):
        call(*a, workspace=torch.empty(1 << 20, dtype=torch.uint8, device="meta"))
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        call(*a, workspace=torch.empty(1 << 20, dtype=torch.uint8)[::2])
    with pytest.raises(TypeError, match="workspace"):
        call(*a, workspace=1 << 20)


@pytest.mark.gpu
@both
def test_two_calls_at_once(dtype):
    """Two streams, each with a workspace of its own, cut sequences among them: what each gives alone."""
    xs = [make([4500, 64], 1, 2, 64, 64, dtype, 40 + i) for i in range(2)]
    ds = [to(x) for x, _ in xs]
    c = torch.tensor(xs[0][1], dtype=torch.int32, device=DEV)

    def both_passes(d, stream):
        a = [d[k] for k in ("q", "k", "v", "g", "beta")]
        o, S = kda.kda_gdr_chunk_fwd(*a, d["S0"], cu_seqlens=c, scale=1.0, stream=stream)
        g = kda.kda_gdr_chunk_bwd(*a, d["do"], d["S0"], d["dS_T"], cu_seqlens=c, scale=1.0, stream=stream)
        return [o, S] + [g[k] for k in sorted(g)]

    want = []
    for d in ds:
        want.append(both_passes(d, None))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    got = [both_passes(d, s) for d, s in zip(ds, streams)]
    torch.cuda.synchronize()
    for p, q in zip(want, got):
        for j, (u, v) in enumerate(zip(p, q)):
            assert torch.equal(u, v), j


@pytest.mark.gpu
def test_two_graphs_share_a_workspace():
    """Two captured calls of different sizes on one workspace, replayed in turn on one stream; the
    workspace holds NaN before the first, and one byte too few is refused."""
    xs = [make([4500], 1, 2, 64, 64, torch.bfloat16, 50), make([70, 9], 1, 2, 64, 64, torch.bfloat16, 51)]
    ds = [(to(x), torch.tensor(cu, dtype=torch.int32, device=DEV)) for x, cu in xs]
    need = max(kda.kda_gdr_chunk_bwd_workspace_size(len(cu) - 1, cu[-1], 2, 64, 64, True) for _, cu in xs)
    ws = torch.full((need // 4,), float("nan"), device=DEV)

    def call(d, c, w):
        a = [d[k] for k in ("q", "k", "v", "g", "beta")]
        o, S = kda.kda_gdr_chunk_fwd(*a, d["S0"], cu_seqlens=c, scale=1.0, workspace=w)
        g = kda.kda_gdr_chunk_bwd(*a, d["do"], d["S0"], d["dS_T"], cu_seqlens=c, scale=1.0, workspace=w)
        return [o, S] + [g[k] for k in sorted(g)]

    with pytest.raises(kda.KdaError):
        call(*ds[0], ws.view(torch.uint8)[:-1])
    want = [call(d, c, None) for d, c in ds]
    torch.cuda.synchronize()
    graphs, got = [], []
    for d, c in ds:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            got.append(call(d, c, ws))
        graphs.append(gr)
    for turn in range(3):
        for i, gr in enumerate(graphs):
            gr.replay()
            torch.cuda.synchronize()
            for j, (u, v) in enumerate(zip(want[i], got[i])):
                assert torch.equal(u, v), (turn, i, j)


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [[0, 7], [3, 3, 9], [5, 11], [9, 9], [12, 12], [0, 0], [-4, 30], [8, 2]])
def test_clear_rows(cu):
    """Rows before the first and behind the last sequence, in rows of 8, 12, 16 and 64 bytes; offsets are held to
    the tensors, and the guard around them stays."""
    T = 12
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    lo = min(max(cu[0], 0), T)
    hi = min(max(cu[-1], lo), T)
    flat = [torch.full((8 * n + T * n + 8 * n,), 3.0, device=DEV) for n in (2, 4, 16, 3)]
    views = [f[8 * n:8 * n + T * n].view(1, T, n) for f, n in zip(flat, (2, 4, 16, 3))]
    kda.kda_gdr_clear_rows(c, *views)
    torch.cuda.synchronize()
    for f, n in zip(flat, (2, 4, 16, 3)):
        assert (f[:8 * n] == 3).all() and (f[8 * n + T * n:] == 3).all()
    for v in views:
        assert (v[0, :lo] == 0).all() and (v[0, hi:] == 0).all() and (v[0, lo:hi] == 3).all()


@pytest.mark.gpu
def test_made_outputs_are_zero_outside_sequences():
    """What the binding makes itself is zero in the rows of no sequence, whatever the memory held."""
    x, cu = make([40, 9], 1, 2, 32, 32, torch.bfloat16, 70, head=6, tail=5)
    for d in (6.0, 7.0):   # memory that the allocator hands out again
        junk = [torch.full_like(x["v"], d, device=DEV) for _ in range(12)]
        del junk
    o, _ = run_fwd(x, cu, 1.0)
    g = run_bwd(x, cu, 1.0)
    for t in (o, *(g[k] for k in ("dq", "dk", "dv", "dg", "dbeta"))):
        assert (t[0, :6] == 0).all() and (t[0, cu[-1]:] == 0).all()


def test_clear_rows_refusals(lib):
    p = (ctypes.c_void_p * 9)(*[(1 << 40) + (i << 28) for i in range(9)])
    n = (ctypes.c_size_t * 9)(*[64] * 9)
    cu = ctypes.c_void_p(1 << 39)
    f = lib.kda_gdr_clear_rows
    assert f(0, 8, cu, 1, p, n, None) == 2 and f(1, 0, cu, 1, p, n, None) == 2
    assert f(1, 8, cu, 0, p, n, None) == 2 and f(1, 8, cu, 9, p, n, None) == 2
    assert f(1, 8, None, 1, p, n, None) == 1 and f(1, 8, cu, 1, None, n, None) == 1 and f(1, 8, cu, 1, p, None, None) == 1
    for bad in (0, 2, 66, 1 << 31):
        assert f(1, 8, cu, 1, p, (ctypes.c_size_t * 1)(bad), None) == 2
    assert f(1, 8, cu, 1, (ctypes.c_void_p * 1)(None), n, None) == 1
    assert f(1, 8, cu, 1, (ctypes.c_void_p * 1)((1 << 40) + 4), n, None) == 4
    assert f(1, 8, cu, 2, (ctypes.c_void_p * 2)(1 << 40, (1 << 40) + 256), n, None) == 6
    t, c = torch.zeros(1, 8, 4), torch.tensor([0, 8], dtype=torch.int32)
    for bad in ((t[0],), (t, torch.zeros(1, 9, 4)), (), (t,)):   # no leading 1, another T, none, not on the GPU
        with pytest.raises(ValueError):
            kda.kda_gdr_clear_rows(c, *bad)
    with pytest.raises(TypeError):
        kda.kda_gdr_clear_rows(c.long(), t)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Hk,Hv,dk,dv", [([1500], 16, 48, 32, 128), ([900, 900], 24, 24, 64, 96), ([1300], 40, 40, 128, 256)])
def test_cut_sequences_of_many_heads(lens, Hk, Hv, dk, dv):
    """Enough heads that the maps take two column tiles a wavefront, the value columns ending inside its
    256; three heads are looked at."""
    x, cu = make(lens, Hk, Hv, dk, dv, torch.bfloat16, sum(lens) + dv, gmu=-5.0)
    o, S_T = run_fwd(x, cu, dk ** -0.5)
    rep = Hv // Hk
    for h in (0, Hv // 2 + 1, Hv - 1):
        y = {k: v[:, :, h // rep:h // rep + 1] if k in ("q", "k") else v[:, :, h:h + 1] for k, v in x.items() if k not in ("S0", "dS_T")}
        y["S0"], y["dS_T"] = x["S0"][:, h:h + 1], x["dS_T"][:, h:h + 1]
        o64, S64, _ = reference(y, cu, dk ** -0.5, False)
        near(o[:, :, h:h + 1], o64, torch.bfloat16, FWD[torch.bfloat16], f"o of head {h}")
        near(S_T[:, h:h + 1], S64, torch.float32, FWD[torch.bfloat16], f"S_T of head {h}")


@pytest.mark.gpu
@both
def test_growing_state(dtype):
    """Positive g is used as it is.  Each token multiplies an earlier error by at most e^g, so over a
    sequence the bounds grow by e^(sum g) = e at most."""
    x, cu = make([100], 1, 2, 64, 64, dtype, 80)
    x["g"] = torch.full_like(x["g"], 0.01)
    grow = 2.72
    o64, S64, g64 = reference(x, cu, 1.0, True)
    o, S_T = run_fwd(x, cu, 1.0)
    near(o, o64, dtype, grow * FWD[dtype], "o")
    near(S_T, S64, torch.float32, grow * FWD[dtype], "S_T")
    g = run_bwd(x, cu, 1.0)
    for k in ("dq", "dk", "dv", "dg", "dbeta", "dS0"):
        near(g[k], g64[k], dtype if k in ("dq", "dk", "dv") else torch.float32, 2 * grow * FWD[dtype], k)


@pytest.mark.gpu
def test_thousands_of_short_sequences_beside_a_long_one():
    """5,000 sequences of 0 to 3 tokens around one of 2,000 that is cut; some are looked at."""
    lens = [i % 4 for i in range(2500)] + [2000] + [(3 * i) % 4 for i in range(2500)]
    x, cu = make(lens, 1, 1, 32, 32, torch.bfloat16, 81)
    o, S_T = run_fwd(x, cu, 0.3)
    g = run_bwd(x, cu, 0.3)
    for i in (0, 1, 63, 64, 2499, 2500, 2501, 4999, 5000):
        a = slice(cu[i], cu[i + 1])
        y = {k: v[:, a] for k, v in x.items() if k not in ("S0", "dS_T")}
        y["S0"], y["dS_T"] = x["S0"][i:i + 1], x["dS_T"][i:i + 1]
        o64, S64, g64 = reference(y, [0, lens[i]], 0.3, True)
        if lens[i]:
            near(o[:, a], o64, torch.bfloat16, FWD[torch.bfloat16], f"o {i}")
            for k in ("dq", "dk", "dv", "dg", "dbeta"):
                near(g[k][:, a], g64[k], torch.bfloat16 if k in ("dq", "dk", "dv") else torch.float32, 2 * FWD[torch.bfloat16], f"{k} {i}")
        near(S_T[i:i + 1], S64, torch.float32, FWD[torch.bfloat16], f"S_T {i}")
        near(g["dS0"][i:i + 1], g64["dS0"], torch.float32, 2 * FWD[torch.bfloat16], f"dS0 {i}")


@pytest.mark.gpu
@both
@pytest.mark.parametrize("lens,Hk,Hv,dk,dv", [
    ([13, 268], 2, 2, 32, 128), ([88, 1], 1, 4, 128, 64), ([257], 2, 4, 32, 128), ([1500], 1, 2, 64, 64), ([700, 1217], 1, 2, 128, 96)])
def test_fp32_results_keep_fp32_precision(lens, Hk, Hv, dk, dv, dtype):
    """The last state and the gradients of g, beta and the start state are fp32 whatever the storage,
    and so is their precision, sequences cut in pieces among them; in the 2-norm, relative.  An
    operand in three bf16 parts leaves 2^-27 of itself and its products leave out 2^-26 (the bounds at the top
    of this file allow for two parts), less than the
    accumulators' rounding of 2^-24.  Eight products one behind another, each a sum of at most 128 terms with one
    rounding a term, their signs independent: sqrt(8 * 128) * 2^-24 / sqrt(3) = 1.1e-6.  dS0 runs through both chains:
    sqrt(2) times that.  dg and dbeta are differences of sums twice their size besides: 2 sqrt(2) times."""
    unit = (8 * 128 / 3) ** 0.5 * 2.0 ** -24
    x, cu = make(lens, Hk, Hv, dk, dv, dtype, 90 + sum(lens), gmu=-4.0)
    print(f"gdr precision lens={lens} {Hk} {Hv} {dk} {dv} {dtype}", flush=True)
    _, S64, g64 = reference(x, cu, dk ** -0.5, True)
    got = dict(run_bwd(x, cu, dk ** -0.5), S_T=run_fwd(x, cu, dk ** -0.5)[1])
    off = {}
    for k, want, times in (("S_T", S64, 1.0), ("dS0", g64["dS0"], 2 ** 0.5), ("dg", g64["dg"], 8 ** 0.5), ("dbeta", g64["dbeta"], 8 ** 0.5)):
        e = float((got[k].double().cpu() - want).norm() / want.norm())
        if not e <= times * unit:
            off[k] = f"{e:.2e} > {times * unit:.2e}"
    assert not off, off


def one_row_view(*shape, dtype=torch.float32, device="cpu", fill=3.0):
    """(a contiguous view of one row [1, 1, *shape] whose row stride is five rows, the memory around it)"""
    big = torch.full((1, 5, *shape), fill, dtype=dtype, device=device)
    t = big[:, ::5]
    assert t.is_contiguous() and t.shape == (1, 1, *shape) and t.stride(1) != big.stride(1)
    return t, big


def test_row_bytes_of_one_row_views(monkeypatch):
    """The stride of an axis of one says nothing of a row's size: what the library is told to clear is the tensor."""
    seen = []

    class Lib:
        @staticmethod
        def kda_gdr_clear_rows(n, T, cu, k, ptrs, sizes, st):
            seen.extend(sizes)
            return 0

    monkeypatch.setattr(kda, "load_library", lambda: Lib)
    t, _ = one_row_view(4, 8)
    none = torch.zeros(1, 1, 6).as_strided((1, 1, 6), (6, 0, 1))
    kda._clear_rows(1, 1, torch.tensor([0, 0], dtype=torch.int32), (t, none, torch.zeros(1, 1, 2, dtype=torch.bfloat16)), None)
    kda._clear_rows(1, 3, torch.tensor([0, 0], dtype=torch.int32), (torch.zeros(1, 3, 4, 8),), None)
    assert seen == [128, 24, 4, 128]


@pytest.mark.gpu
def test_one_row_views_keep_what_is_around():
    """Clearing, and a backward pass whose gradients are made with the inputs' strides."""
    cu = torch.tensor([0, 0], dtype=torch.int32, device=DEV)
    t, big = one_row_view(4, 8, device=DEV)
    kda.kda_gdr_clear_rows(cu, t)
    torch.cuda.synchronize()
    assert (big[:, 0] == 0).all() and (big[:, 1:] == 3).all()
    q, v = (one_row_view(2, 32, dtype=torch.bfloat16, device=DEV, fill=0.5)[0] for _ in range(2))
    g = one_row_view(2, device=DEV, fill=-0.5)[0]
    d = kda.kda_gdr_chunk_bwd(q, q, v, g, g, v, cu_seqlens=cu, scale=1.0)
    torch.cuda.synchronize()
    for k in ("dq", "dk", "dv", "dg", "dbeta"):
        assert d[k].shape[:2] == (1, 1) and not d[k].any(), k


@pytest.mark.parametrize("nseq,T,Hv", [(4096, 262144, 16), (1024, 65536, 8), (8000, 65536, 4), (100000, 2000000, 1), (3, 65536, 16), (600, 9000, 2), (1, 65536, 32)])
def test_workspace_of_many_packed_sequences(lib, nseq, T, Hv):
    """Beside what every chunk takes, the maps and states of pieces: pieces are cut for 256 compute units, and
    sequences that are not cut have none, however many they are.  Rows hold at most 256 / heads whole pieces, and twice
    that many places are enough."""
    dk = dv = 128
    chunks = (T // 64 + nseq) * Hv
    one, two = kda.kda_gdr_chunk_fwd_workspace_size(1, 64, 1, dk, dv), kda.kda_gdr_chunk_bwd_workspace_size(1, 64, 1, dk, dv)
    f = kda.kda_gdr_chunk_fwd_workspace_size(nseq, T, Hv, dk, dv, True) - chunks * one
    b = kda.kda_gdr_chunk_bwd_workspace_size(nseq, T, Hv, dk, dv, True) - chunks * two
    assert 0 <= f <= 512 * 4 * (dk * (dv + dk) + dk * dv)
    assert 0 <= b <= 512 * 4 * (dk * (dv + dk) + 3 * dk * dv)


MANY = [i % 4 for i in range(400)] + [4500] + [(3 * i) % 4 for i in range(300)] + [2500, 2300, 1, 2700] + [1] * 300


@pytest.mark.gpu
@both
@pytest.mark.parametrize("Hk,Hv,dk,dv", [(1, 2, 64, 64), (1, 1, 32, 96)])
def test_cut_sequences_among_a_thousand_short_ones(Hk, Hv, dk, dv, dtype):
    """More sequences than pieces fit the rows: three are cut, one long one is not; those and some short ones are looked at."""
    x, cu = make(MANY, Hk, Hv, dk, dv, dtype, 95 + dv, head=3, tail=70, gmu=-5.0)
    print(f"gdr many {Hk} {Hv} {dk} {dv} {dtype}", flush=True)
    o, S_T = run_fwd(x, cu, 0.3)
    g = run_bwd(x, cu, 0.3)
    for i in (0, 3, 399, 400, 401, 699, 700, 701, 702, 703, 704, 705, 1003):
        a = slice(cu[i], cu[i + 1])
        y = {k: v[:, a] for k, v in x.items() if k not in ("S0", "dS_T")}
        y["S0"], y["dS_T"] = x["S0"][i:i + 1], x["dS_T"][i:i + 1]
        o64, S64, g64 = reference(y, [0, MANY[i]], 0.3, True)
        near(S_T[i:i + 1], S64, torch.float32, FWD[dtype], f"S_T {i}")
        near(g["dS0"][i:i + 1], g64["dS0"], torch.float32, 2 * FWD[dtype], f"dS0 {i}")
        if MANY[i]:
            near(o[:, a], o64, dtype, FWD[dtype], f"o {i}")
            for k in ("dq", "dk", "dv", "dg", "dbeta"):
                near(g[k][:, a], g64[k], dtype if k in ("dq", "dk", "dv") else torch.float32, 2 * FWD[dtype], f"{k} {i}")
    S = x["S0"].to(DEV)   # and the last states written over the start states
    d = to(x)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    o2, _ = kda.kda_gdr_chunk_fwd(*(d[k] for k in ("q", "k", "v", "g", "beta")), S, cu_seqlens=c, S_T=S, scale=0.3)
    assert torch.equal(o, o2) and torch.equal(S, S_T)


@pytest.mark.gpu
def test_many_offsets_out_of_order_touch_nothing_else():
    """As above with so many sequences that pieces have places of their own: the tensors and a workspace of just the
    size asked for keep the guards around them."""
    rows, n, Hv = 9000, 600, 1
    x, _ = make([rows], 1, Hv, 32, 32, torch.bfloat16, 96)
    d = to(x)
    a = [d[k] for k in ("q", "k", "v", "g", "beta")]
    pad = torch.full((rows + 256, Hv, 32), 5.0, dtype=torch.bfloat16, device=DEV)
    o = pad[128:128 + rows].unsqueeze(0)
    need = kda.kda_gdr_chunk_bwd_workspace_size(n, rows, Hv, 32, 32, True)
    mem = torch.full((need + (1 << 21),), 9, dtype=torch.uint8, device=DEV)
    ws = mem[1 << 20:(1 << 20) + need]
    gen = torch.Generator().manual_seed(5)
    for cu in ([0] + [rows] * n, [0, rows] * 300 + [0], [rows] * n + [0], torch.randint(-rows, 2 * rows, (n + 1,), generator=gen).tolist(),
               torch.randint(0, rows + 1, (n + 1,), generator=gen).tolist()):
        c = torch.tensor(cu, dtype=torch.int32, device=DEV)
        kda.kda_gdr_chunk_fwd(*a, cu_seqlens=c, scale=1.0, o=o, workspace=ws)
        kda.kda_gdr_chunk_bwd(*a, d["do"], cu_seqlens=c, scale=1.0, workspace=ws)
        torch.cuda.synchronize()
        assert (pad[:128] == 5).all() and (pad[128 + rows:] == 5).all(), cu[:4]
        assert (mem[:1 << 20] == 9).all() and (mem[(1 << 20) + need:] == 9).all(), cu[:4]


@pytest.mark.gpu
def test_cut_sequence_among_half_a_million():
    """2^19 sequences, 256 columns: joins for every sequence would be 2^32 threads; only those that may be
    cut have any.  One holds all the rows and is cut; alone it is cut elsewhere, so both are off by the
    tolerance at most."""
    n, rows = 1 << 19, 64 * 30000
    gen = torch.Generator(device=DEV).manual_seed(3)
    r = lambda *s, dt=torch.bfloat16: torch.randn(*s, generator=gen, device=DEV, dtype=dt)   # noqa: E731
    q, k = (torch.nn.functional.normalize(r(1, rows, 1, 32), dim=-1) for _ in range(2))
    v, g, beta = r(1, rows, 1, 256), -0.02 * r(1, rows, 1, dt=torch.float32).abs(), torch.sigmoid(r(1, rows, 1, dt=torch.float32))
    cu = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    cu[n // 2 + 7:] = rows
    S0 = 0.2 * r(1, 1, 32, 256, dt=torch.float32)
    states = torch.zeros(n, 1, 32, 256, device=DEV)
    states[n // 2 + 6] = S0[0]
    print(f"gdr {n} sequences, {rows} rows", flush=True)
    o, S = kda.kda_gdr_chunk_fwd(q, k, v, g, beta, states, cu_seqlens=cu, scale=1.0)
    o2, S2 = kda.kda_gdr_chunk_fwd(q, k, v, g, beta, S0, scale=1.0)
    torch.cuda.synchronize()
    assert torch.equal(S[:n // 2 + 6], states[:n // 2 + 6]) and torch.equal(S[n // 2 + 7:], states[n // 2 + 7:])
    near(S[n // 2 + 6:n // 2 + 7], S2.double().cpu(), torch.float32, 2 * FWD[torch.bfloat16], "S_T")
    near(o, o2.double().cpu(), torch.bfloat16, 2 * FWD[torch.bfloat16] + 2 * HALF_STEP[torch.bfloat16], "o")
