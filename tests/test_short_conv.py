"""kda_short_conv_fwd, _bwd and _step against the definition in 64 bits.

Tolerance: a pre-activation is a sum of W products and a bias in fp32, at most W + 1 roundings of the
sum of their sizes m.  In fp32 storage silu adds 8 (the sigmoid's exponential and division, the product), and carries
a pre-activation's error by a slope of at most 1.1; in bf16 storage the sigmoid comes from the hardware exponential of a rounded argument, whose
error of |p| roundings is added.  So y is off by at most 1.1 (W + 1) + 8 + 2 |p| roundings of m.  A dp has those of
its pre-activation through silu'' (at most 0.5), of silu' itself and of a product: 2 W + 16 + 3 |p| of |dy| max(1, m);
dx and dS0 are sums of W of them, dw and dbias of T (a product and a sum each), of magnitudes summed the same way.
"""
import ctypes

import pytest
import torch

import chunked_gated_delta_12_amd as kda
from plain_ops import close
from plain_state_space import conv64

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def inputs(B, T, D, W, dtype, seed, bias=True, n=None, S0=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    return dict(x=r(B, T, D).to(dtype), w=(2 * torch.rand(D, W, generator=gen) - 1) * W ** -0.5, bias=0.1 * r(D) if bias else None,
                S0=r(n or B, W - 1, D).to(dtype) if S0 else None)


def to_dev(x):
    return {k: None if v is None else v.to(DEV) for k, v in x.items()}


def spans(B, T, lens, first=0):
    if lens is None:
        return [(i, 0, T) for i in range(B)]
    out, lo = [], first
    for n in lens:
        out.append((0, lo, lo + n))
        lo += n
    return out


def cu_of(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def sequence(x, i, lo, hi, n):
    W, D = x["w"].shape[1], x["w"].shape[0]
    S = torch.zeros(W - 1, D).double() if x["S0"] is None else x["S0"][n].double()
    return x["x"][i, lo:hi].double(), x["w"].double(), None if x["bias"] is None else x["bias"].double(), S


def sizes(xs, w, bias, S):
    return conv64(xs.abs(), w.abs(), None if bias is None else bias.abs(), S.abs(), None)[0]


def check_fwd(x, y, S_T, sp, act, dtype):
    W = x["w"].shape[1]
    for n, (i, lo, hi) in enumerate(sp):
        a = sequence(x, i, lo, hi, n)
        y64, S64 = conv64(*a, act)
        m = sizes(*a)
        close(y[i, lo:hi], y64, dtype, m * (1.1 * (W + 1) + 8 + 2 * m), 1, f"y of sequence {n}")
        if S_T is not None:
            assert torch.equal(S_T[n].double(), S64), n


LENS = [5, 0, 1, 2, 40, 3, 0, 0, 33, 64]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("B,T,D,W,S0", [(1, 1, 8, 4, True), (2, 2, 24, 4, False), (3, 33, 520, 3, True), (1, 100, 2056, 2, True), (1, LENS, 40, 4, True),
                                        (1, LENS, 512, 3, False), (1, [1000, 1, 1500], 64, 4, True)])
def test_fwd_and_bwd(B, T, D, W, S0, act, dtype):
    print(f"conv B={B} T={T} D={D} W={W} S0={S0} act={act} {dtype}", flush=True)
    lens, rows = (T, sum(T)) if isinstance(T, list) else (None, T)
    n = len(lens) if lens else B
    x = inputs(B, rows, D, W, dtype, 3, bias=D != 24, n=n, S0=S0)
    d, cu = to_dev(x), cu_of(lens) if lens else None
    sp = spans(B, rows, lens)
    y, S_T = kda.kda_short_conv_fwd(d["x"], d["w"], d["S0"], bias=d["bias"], act=act, cu_seqlens=cu)
    torch.cuda.synchronize()
    check_fwd(x, y.cpu(), S_T.cpu(), sp, act, dtype)
    gen = torch.Generator().manual_seed(5)
    dy = torch.randn(B, rows, D, generator=gen).to(dtype)
    dS = torch.randn(n, W - 1, D, generator=gen).to(dtype) if S0 else None
    got = kda.kda_short_conv_bwd(d["x"], d["w"], dy.to(DEV), d["S0"], None if dS is None else dS.to(DEV), bias=d["bias"], act=act, cu_seqlens=cu)
    torch.cuda.synchronize()
    check_bwd(got, x, dy, dS, sp, act, dtype)


def check_bwd(got, x, dy, dS, sp, act, dtype):
    D, W = x["w"].shape
    dw, db = torch.zeros(D, W).double(), torch.zeros(D).double()
    mw, mb, most, rows = torch.zeros_like(dw), torch.zeros_like(db), 0.0, 0
    for n, (i, lo, hi) in enumerate(sp):
        xs, w, bias, S = sequence(x, i, lo, hi, n)
        leaves = [t.requires_grad_() for t in (xs, w, S) + (() if bias is None else (bias,))]
        y, S_T = conv64(xs, w, bias, S, act)
        gy = dy[i, lo:hi].double()
        loss = (y * gy).sum() + (0 if dS is None else (S_T * dS[n].double()).sum()) + 0 * w.sum()
        g = [torch.zeros_like(v) if t is None else t for v, t in zip(leaves, torch.autograd.grad(loss, leaves, allow_unused=True))]
        m = sizes(*(t if t is None else t.detach() for t in (xs, w, bias, S)))
        # a dp's error in roundings, and its own size
        e = gy.abs() * (2 * W + 16 + 3 * m) * m.clamp_min(1)
        pads = [t.detach().abs().requires_grad_() for t in (xs, w, S)]
        for err in (e, gy.abs() * 1.1):   # what sums of W, or of all rows, of them are off by; the sums' own roundings
            yl, sl = conv64(*pads[:2], None, pads[2], None)
            l2 = (yl * err).sum() + (0 if dS is None else (sl * dS[n].double().abs()).sum()) + 0 * pads[1].sum()
            gm = [torch.zeros_like(v) if t is None else t for v, t in zip(pads, torch.autograd.grad(l2, pads, allow_unused=True))]
            if err is e:
                mx, ms, mwn = gm[0], gm[2], gm[1]
            else:
                mx, ms, mwn = mx + (W + 2) * gm[0], ms + (W + 2) * gm[2], mwn + (hi - lo + 40) * gm[1]
        close(got["dx"][i, lo:hi], g[0], dtype, mx, 1, f"dx of sequence {n}")
        close(got["dS0"][n], g[2], dtype, ms, 1, f"dS0 of sequence {n}")
        dw += g[1]
        mw += mwn
        if bias is not None:
            db += g[3]
            mb += e.sum(0) + (hi - lo + 40) * 1.1 * gy.abs().sum(0)
    rows = sum(hi - lo for _, lo, hi in sp)
    close(got["dw"], dw, F32, mw * (1 + len(sp) / max(1, rows)), 1, "dw")
    if x["bias"] is not None:
        close(got["dbias"], db, F32, mb * (1 + len(sp) / max(1, rows)), 1, "dbias")
    else:
        assert got["dbias"] is None


def test_plain_gradients_against_differences():
    gen = torch.Generator().manual_seed(0)
    x, w, b, S = (torch.randn(*s, generator=gen).double().requires_grad_() for s in ((6, 8), (8, 4), (8,), (3, 8)))
    assert torch.autograd.gradcheck(lambda *a: conv64(*a, "silu"), (x, w, b, S))


@pytest.mark.gpu
def test_linear_gradient_is_the_transpose():
    """Without an activation <dy, conv(x)> = <conv^T(dy), x> for the kernels' own results: in fp32 both sums differ by at
    most W + 2 roundings of the sum of all sizes."""
    B, T, D, W = 2, 77, 40, 4
    x = inputs(B, T, D, W, F32, 1, bias=False, S0=False)
    d = to_dev(x)
    dy = torch.randn(B, T, D, generator=torch.Generator().manual_seed(2)).to(DEV)
    y, _ = kda.kda_short_conv_fwd(d["x"], d["w"])
    g = kda.kda_short_conv_bwd(d["x"], d["w"], dy)
    mag = sum((sizes(x["x"][i].double(), x["w"].double(), None, torch.zeros(W - 1, D).double()) * dy[i].double().cpu().abs()).sum() for i in range(B))
    left, right = (y.double() * dy.double()).sum().item(), (g["dx"].double() * d["x"].double()).sum().item()
    assert abs(left - right) <= 2 * (W + 2) * U * mag


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_no_sequence(dtype):
    D, W, lens, first, rows = 24, 4, [40, 0, 70], 3, 120
    x = inputs(1, rows, D, W, dtype, 9, n=3)
    none = torch.ones(rows, dtype=torch.bool)
    none[first:first + sum(lens)] = False
    x["x"][0, none] = float("nan")
    d, cu, sp = to_dev(x), cu_of(lens, first), spans(1, rows, lens, first)
    kept = torch.full((1, rows, D), 5.0, dtype=dtype, device=DEV)
    y, S_T = kda.kda_short_conv_fwd(d["x"], d["w"], d["S0"], bias=d["bias"], act="silu", cu_seqlens=cu, y=kept)
    check_fwd(x, y.cpu(), S_T.cpu(), sp, "silu", dtype)
    assert (y.cpu()[0, none] == 5).all()
    y, _ = kda.kda_short_conv_fwd(d["x"], d["w"], d["S0"], bias=d["bias"], act="silu", cu_seqlens=cu)
    assert not y.cpu()[0, none].any()
    dy = torch.randn(1, rows, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    dy[0, none] = float("nan")
    got = kda.kda_short_conv_bwd(d["x"], d["w"], dy.to(DEV), d["S0"], bias=d["bias"], act="silu", cu_seqlens=cu)
    assert not got["dx"].cpu()[0, none].any()
    check_bwd(got, x, dy, None, sp, "silu", dtype)


@pytest.mark.gpu
def test_offsets_out_of_order_stay_inside():
    D, W, rows = 64, 4, 300
    x = inputs(1, rows, D, W, F32, 2, n=4)
    d = to_dev(x)
    cu = torch.tensor([50, 10, -7, 1 << 30, 20], dtype=torch.int32, device=DEV)
    big, S = torch.full((3, rows, D), 2.0, device=DEV), torch.full((3, 4, W - 1, D), 2.0, device=DEV)
    kda.kda_short_conv_fwd(d["x"], d["w"], d["S0"], cu_seqlens=cu, y=big[1:2], S_T=S[1])
    kda.kda_short_conv_bwd(d["x"], d["w"], big[1:2], d["S0"], cu_seqlens=cu)
    torch.cuda.synchronize()
    for t in (big[0], big[2], S[0], S[2]):
        assert (t == 2).all()


@pytest.mark.gpu
def test_state_in_place_and_pieces():
    """Sequences in two calls, the state written over itself, equal one call bit for bit: each output is the same sum."""
    D, W = 40, 4
    for lens, cut in (([2, 1, 9], [1, 0, 6]), ([70, 3, 40], [33, 2, 0])):
        x = inputs(1, sum(lens), D, W, BF16, 4, n=3)
        d = to_dev(x)
        y, S_T = kda.kda_short_conv_fwd(d["x"], d["w"], d["S0"], act="silu", cu_seqlens=cu_of(lens))
        S, halves = d["S0"].clone(), []
        for part in (0, 1):
            rows, ls = [], []
            for (_, lo, hi), c in zip(spans(1, 0, lens), cut):
                lo, hi = (lo, lo + c) if part == 0 else (lo + c, hi)
                rows += list(range(lo, hi))
                ls.append(hi - lo)
            yp, S2 = kda.kda_short_conv_fwd(d["x"][:, rows].contiguous(), d["w"], S, act="silu", cu_seqlens=cu_of(ls), S_T=S)
            assert S2 is S
            halves.append((rows, yp))
        for rows, yp in halves:
            assert torch.equal(yp[0], y[0, rows])
        assert torch.equal(S, S_T)


def step(x, slots, ntok, act, y=None):
    d = to_dev(x)
    t = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)   # noqa: E731
    y = kda.kda_short_conv_step(d["x"], d["w"], d["S0"], bias=d["bias"], act=act, slots=t(slots), ntok=t(ntok), y=None if y is None else y.to(DEV))
    torch.cuda.synchronize()
    return y.cpu(), d["S0"].cpu()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,D,W", [(1, 1, 8, 4), (3, 1, 520, 2), (2, 5, 72, 3), (2, 9, 1032, 4)])
def test_step(B, T, D, W, dtype):
    x = inputs(B, T, D, W, dtype, 6)
    y, S = step(x, None, None, "silu")
    check_fwd(x, y, S, spans(B, T, None), "silu", dtype)


@pytest.mark.gpu
def test_step_slots_padding_and_duplicates():
    B, T, D, W, P = 9, 3, 40, 4, 12
    x = inputs(B, T, D, W, BF16, 3, n=P)
    slots = [5, -1, 0, 11, 5, 12, 7, 2, 1 << 30]
    ntok = [0, 3, 1, 9, 3, 2, 0, 2, 1]
    real = {2: 1, 3: 3, 4: 3, 7: 2}
    y0 = torch.full((B, T, D), 7.0).to(BF16)
    y, S = step(x, slots, ntok, "silu", y0)
    for b, n in real.items():
        one = dict(x, S0=x["S0"][slots[b]][None], x=x["x"][b:b + 1, :n])
        check_fwd(one, y[b:b + 1, :n], S[slots[b]][None], [(0, 0, n)], "silu", BF16)
        assert torch.equal(y[b, n:], y0[b, n:])
    for b in set(range(B)) - set(real):
        assert torch.equal(y[b], y0[b]), b
    for s in set(range(P)) - {slots[b] for b in real}:
        assert torch.equal(S[s], x["S0"][s]), s


@pytest.mark.gpu
def test_graph_and_not_finite():
    T, D, W = 200, 64, 4
    x = [to_dev(inputs(1, T, D, W, BF16, s)) for s in (1, 2)]
    x[1]["x"][0, 50, 3] = float("inf")
    dy = torch.randn(1, T, D, device=DEV).to(BF16)
    st = {k: v.clone() for k, v in x[0].items()}

    def call(a):
        y, S = kda.kda_short_conv_fwd(a["x"], a["w"], a["S0"], bias=a["bias"], act="silu")
        g = kda.kda_short_conv_bwd(a["x"], a["w"], dy, a["S0"], bias=a["bias"], act="silu")
        return [y, S, g["dx"], g["dw"], g["dbias"], g["dS0"]]

    call(st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(st)
    for i in (0, 1, 0, 1):
        for k, v in st.items():
            v.copy_(x[i][k])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, call(x[i])):
            assert torch.equal(torch.nan_to_num(a, nan=9.0), torch.nan_to_num(b, nan=9.0))
    bad = ~torch.isfinite(out[0][0])
    assert bad[50:54, 3].any() and not bad[:50].any() and not bad[54:].any() and not bad[:, :3].any() and not bad[:, 4:].any()


# ----------------------------------------------------------------------------- refusals (no GPU)
@pytest.fixture(scope="module")
def lib():
    try:
        return kda.load_library()
    except RuntimeError as e:
        pytest.skip(str(e))


NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, ALIAS = 1, 2, 3, 4, 5, 6
AT = {k: (1 << 40) + (i << 30) for i, k in enumerate("cu x w bias S0 dy dS_T y S_T dx dw dbias dS0 ws slots ntok".split())}


def call(lib, which, **over):
    v = dict(dtype=0, act=1, rest=1, n=2, T=64, D=64, W=4, nslot=4, bytes=1 << 29)
    v.update(AT)
    v["cu"] = None
    v.update(over)
    p = lambda *names: [None if v[n] is None else ctypes.c_void_p(v[n]) for n in names]   # noqa: E731
    head = [v[k] for k in ("dtype", "act", "n", "T", "D", "W")]
    if which == "fwd":
        return lib.kda_short_conv_fwd(*head, *p("cu"), v["rest"], *p("x", "w", "bias", "S0", "y", "S_T"), None)
    if which == "bwd":
        return lib.kda_short_conv_bwd(*head, *p("cu", "x", "w", "bias", "S0", "dy", "dS_T", "dx", "dw", "dbias", "dS0", "ws"), v["bytes"], None)
    return lib.kda_short_conv_step(*head, v["nslot"], *p("x", "w", "bias", "S0", "slots", "ntok", "y"), None)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=3), DTYPE), (dict(act=2), SHAPE), (dict(act=-1), SHAPE), (dict(n=0), SHAPE), (dict(T=0), SHAPE), (dict(T=(1 << 30) + 1), SHAPE),
    (dict(D=12), SHAPE), (dict(D=0), SHAPE), (dict(D=1 << 21), SHAPE), (dict(W=1), SHAPE), (dict(W=5), SHAPE), (dict(n=1 << 30, T=1 << 20), SHAPE),
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(x=AT["x"] + 2), ALIGN), (dict(bias=AT["bias"] + 8), ALIGN)])
def test_refusals_of_all(lib, over, status):
    for which in ("fwd", "bwd", "step"):
        assert call(lib, which, **over) == status, which


def test_refusals_of_each(lib):
    assert call(lib, "fwd", rest=2) == SHAPE
    assert call(lib, "fwd", y=None) == NULL and call(lib, "bwd", dw=None) == NULL and call(lib, "step", S0=None) == NULL
    assert call(lib, "bwd", bias=None) == NULL
    assert call(lib, "fwd", y=AT["x"]) == ALIAS and call(lib, "fwd", S_T=AT["S0"] + 16) == ALIAS and call(lib, "fwd", S_T=AT["x"]) == ALIAS
    assert call(lib, "bwd", dx=AT["dy"]) == ALIAS and call(lib, "bwd", dS0=AT["S0"]) == ALIAS and call(lib, "bwd", ws=AT["dx"]) == ALIAS
    assert call(lib, "step", y=AT["x"]) == ALIAS and call(lib, "step", S0=AT["y"]) == ALIAS
    assert call(lib, "bwd", ws=None) == WORKSPACE and call(lib, "bwd", bytes=16) == WORKSPACE
    assert call(lib, "step", nslot=0) == SHAPE and call(lib, "step", nslot=1, slots=None) == SHAPE
    size = ctypes.c_size_t(0)
    assert lib.kda_short_conv_bwd_workspace_size(100, 64, 4, None) == NULL
    assert lib.kda_short_conv_bwd_workspace_size(0, 64, 4, ctypes.byref(size)) == SHAPE
    assert lib.kda_short_conv_bwd_workspace_size(100, 64, 4, ctypes.byref(size)) == 0 and size.value >= 64 * 5 * 4


def test_binding_refuses(lib):
    x = inputs(1, 4, 8, 4, F32, 0)
    with pytest.raises(ValueError):   # on the CPU
        kda.kda_short_conv_fwd(x["x"], x["w"])
    with pytest.raises(ValueError):
        kda.kda_short_conv_fwd(x["x"], x["w"], act="relu")
    with pytest.raises(TypeError):
        kda.kda_short_conv_fwd(x["x"], x["w"].double())
    with pytest.raises(ValueError):
        kda.kda_short_conv_fwd(x["x"], x["w"].t().contiguous().t())
    with pytest.raises(ValueError):
        kda.kda_short_conv_fwd(x["x"], x["w"], x["S0"][:, :2])
