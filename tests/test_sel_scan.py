"""kda_sel_scan_fwd, _bwd and _step against the token-by-token definition in 64 bits.

Tolerance: every value is a chain of products and sums in fp32.  A step size is off by at most 8
roundings (the sum with its bias, the exponential 3, the reciprocal 2, the series 2), so a decay
exp(delta A) by 8 |delta A| for the step, 3 |delta A| for A log2 e, the product and its scale, and 3 for the exponential itself;
with the products and sums around it a token adds at most 11 m + 8 roundings, m the largest
|delta A|, to a state's path forwards, and as many to a gradient's path backwards.  What is cut is joined with
a chain that adds no more than the tokens it stands for.  Sums over N states, D channels and T tokens add a
rounding a term.  So values are off by at most T (11 m + 8) + N + 24 roundings forwards and gradients by
2 T (11 m + 8) + T + D + N + 48, of magnitudes taken from the same sums over absolute values; what is
stored in bf16 is rounded once more.
"""
import ctypes
import math

import pytest
import torch

import chunked_gated_delta_12_amd as kda
from plain_ops import close
from plain_state_space import scan64, scan_magnitudes, step_size

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def inputs(B, T, D, N, G, dtype, seed, parts="skip z dt_bias", softplus=True, n=None):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    x = dict(x=r(B, T, D).to(dtype), b=r(B, T, G, N).to(dtype), c=r(B, T, G, N).to(dtype))
    x["A"] = -torch.arange(1, N + 1).float() * torch.exp(0.2 * r(D, N))
    size = torch.exp(torch.rand(D, generator=gen) * math.log(100.0)) * 1e-3
    x["dt"] = (0.5 * r(B, T, D) if softplus else size * torch.exp(0.5 * r(B, T, D))).to(dtype)
    x["dt_bias"] = torch.log(torch.expm1(size)) if "dt_bias" in parts and softplus else None
    x["skip"] = 1 + 0.1 * r(D) if "skip" in parts else None
    x["z"] = r(B, T, D).to(dtype) if "z" in parts else None
    x["S0"] = 0.3 * r(n or B, D, N) if "S0" in parts else None
    return x


def options(x, softplus):
    return dict(skip=x["skip"], z=x["z"], dt_bias=x["dt_bias"], softplus=softplus)


def to_dev(x):
    return {k: None if v is None else v.to(DEV) for k, v in x.items()}


def sequence(x, i, lo, hi, n):
    """The parts of one sequence, in 64 bits."""
    a = {k: None if x[k] is None else x[k][i, lo:hi].double() for k in ("x", "dt", "b", "c", "z")}
    a.update({k: None if x[k] is None else x[k].double() for k in ("A", "skip", "dt_bias")})
    a["S"] = torch.zeros(x["A"].shape).double() if x["S0"] is None else x["S0"][n].double()
    return a


def per_token(a, softplus):
    d = step_size(a["dt"], a["dt_bias"], softplus)
    return 11 * float((d.abs().max() if d.numel() else 0.0) * a["A"].abs().max()) + 8


def spans(B, T, lens):
    """(row of the batch, first, last) of each sequence."""
    if lens is None:
        return [(i, 0, T) for i in range(B)]
    out, lo = [], 0
    for n in lens:
        out.append((0, lo, lo + n))
        lo += n
    return out


def cu_of(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def check_fwd(x, y, S_T, sp, softplus, dtype):
    D, N = x["A"].shape
    for n, (i, lo, hi) in enumerate(sp):
        a = sequence(x, i, lo, hi, n)
        y64, S64 = scan64(a, softplus)
        m = scan_magnitudes(a, softplus)
        r = (hi - lo) * per_token(a, softplus) + N + 24
        close(y[i, lo:hi], y64, dtype, m["y"][:hi - lo], r, f"y of sequence {n}")
        if S_T is not None:
            close(S_T[n], S64, F32, m["S"], r, f"S_T of sequence {n}")


FWD = [  # B, T or lengths, D, N, G, parts, softplus
    (1, 1, 8, 8, 1, "", False), (2, 3, 8, 16, 1, "S0", True), (1, 33, 64, 16, 1, "skip z dt_bias", True), (2, 31, 72, 32, 3, "z S0", False),
    (1, 130, 136, 64, 1, "skip z dt_bias S0", True), (1, [5, 0, 1, 64, 65, 0], 40, 16, 1, "skip z dt_bias S0", True),
    (1, [200, 1, 129], 256, 8, 4, "skip dt_bias S0", True), (1, [0, 0, 3], 16, 16, 2, "z", True), (3, 257, 24, 16, 1, "skip z dt_bias S0", True)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,D,N,G,parts,softplus", FWD)
def test_fwd(B, T, D, N, G, parts, softplus, dtype):
    print(f"scan fwd B={B} T={T} D={D} N={N} G={G} {parts} {dtype}", flush=True)
    lens, rows = (T, sum(T)) if isinstance(T, list) else (None, T)
    x = inputs(B, rows, D, N, G, dtype, 3, parts, softplus, len(lens) if lens else None)
    d = to_dev(x)
    y, S_T = kda.kda_sel_scan_fwd(d["x"], d["dt"], d["A"], d["b"], d["c"], d["S0"], cu_seqlens=cu_of(lens) if lens else None, **options(d, softplus))
    torch.cuda.synchronize()
    check_fwd(x, y.cpu(), S_T.cpu(), spans(B, rows, lens), softplus, dtype)


NAMES = ("dx", "ddt", "dA", "db", "dc", "dskip", "dz", "ddt_bias", "dS0")


def gradients64(x, dy, dS, sp, softplus):
    """(gradients, magnitudes, roundings) of the whole call, in 64 bits."""
    D, N = x["A"].shape
    whole = {n: x[n[1:]] for n in NAMES[:-1]}
    g = {n: None if v is None else torch.zeros(v.shape).double() for n, v in whole.items()}
    g["dS0"] = torch.zeros(len(sp), D, N).double()
    mag, most = {n: None if v is None else v.clone() for n, v in g.items()}, 0.0
    for n, (i, lo, hi) in enumerate(sp):
        a = sequence(x, i, lo, hi, n)
        leaves = {k: v.requires_grad_() for k, v in a.items() if v is not None}
        y, S = scan64(a, softplus)
        gy = dy[i, lo:hi].double()
        gS = None if dS is None else dS[n].double()
        loss = (y * gy).sum() + (0 if gS is None else (S * gS).sum())
        if loss.requires_grad:
            got = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()), allow_unused=True)))
        else:
            got = {}
        m = scan_magnitudes(a, softplus, gy, gS)
        for k in NAMES:
            name = "S" if k == "dS0" else k[1:]
            if g[k] is None:
                continue
            v, w = got.get(name), m[k]
            v = torch.zeros_like(w) if v is None else v
            if k in ("dx", "ddt", "db", "dc", "dz"):
                g[k][i, lo:hi], mag[k][i, lo:hi] = v, w
            elif k == "dS0":
                g[k][n], mag[k][n] = v, w
            else:
                g[k] += v
                mag[k] += w
        most = max(most, (hi - lo) * per_token({k: v.detach() if torch.is_tensor(v) else v for k, v in a.items()}, softplus))
    rows = sum(hi - lo for _, lo, hi in sp)
    return g, mag, 2 * most + rows + D + N + 48


def check_bwd(got, x, dy, dS, sp, softplus, dtype):
    g, mag, r = gradients64(x, dy, dS, sp, softplus)
    for k in NAMES:
        if k == "dS0" and got[k] is None:
            continue
        assert (got[k] is None) == (g[k] is None), k
        if g[k] is not None:
            close(got[k], g[k], got[k].dtype, mag[k], r, k)


BWD = [(1, 1, 8, 8, 1, "", False, False), (2, 3, 8, 16, 1, "S0", True, True), (1, 33, 64, 16, 1, "skip z dt_bias", True, False),
       (2, 31, 72, 32, 3, "z S0", False, True), (1, 130, 72, 64, 1, "skip z dt_bias S0", True, True), (1, [5, 0, 1, 64, 65, 0], 40, 16, 1, "skip z dt_bias S0", True, True),
       (1, [150, 1, 77], 128, 8, 4, "skip dt_bias S0", True, False), (1, [0, 0, 3], 16, 16, 2, "z", True, True), (2, 200, 24, 16, 1, "skip z dt_bias S0", True, True)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,D,N,G,parts,softplus,last", BWD)
def test_bwd(B, T, D, N, G, parts, softplus, last, dtype):
    print(f"scan bwd B={B} T={T} D={D} N={N} G={G} {parts} {dtype}", flush=True)
    lens, rows = (T, sum(T)) if isinstance(T, list) else (None, T)
    n = len(lens) if lens else B
    x = inputs(B, rows, D, N, G, dtype, 4, parts, softplus, n)
    gen = torch.Generator().manual_seed(8)
    dy = torch.randn(B, rows, D, generator=gen).to(dtype)
    dS = 0.3 * torch.randn(n, D, N, generator=gen) if last else None
    d = to_dev(x)
    got = kda.kda_sel_scan_bwd(d["x"], d["dt"], d["A"], d["b"], d["c"], dy.to(DEV), d["S0"], None if dS is None else dS.to(DEV),
                               cu_seqlens=cu_of(lens) if lens else None, **options(d, softplus))
    torch.cuda.synchronize()
    check_bwd(got, x, dy, dS, spans(B, rows, lens), softplus, dtype)


def test_plain_gradients_against_differences():
    """The 64-bit definition's gradients against central differences in 64 bits: with steps of 1e-5 a difference is off
    by 1e-10 of third derivatives (of the loss's own size here, up to some hundreds) and 1e-16 / 1e-5 of the loss."""
    x = inputs(1, 5, 8, 8, 1, F32, 1, "skip z dt_bias S0")
    a = sequence(x, 0, 0, 5, 0)
    gen = torch.Generator().manual_seed(2)
    dy, dS = torch.randn(5, 8, generator=gen).double(), torch.randn(8, 8, generator=gen).double()

    def loss(a):
        y, S = scan64(a, True)
        return (y * dy).sum() + (S * dS).sum()

    leaves = {k: v.clone().requires_grad_() for k, v in a.items()}
    g = torch.autograd.grad(loss(leaves), list(leaves.values()))
    for k, gk in zip(leaves, g):
        v = torch.randn(gk.shape, generator=gen).double()
        up, down = (loss(dict(a, **{k: a[k] + s * 1e-5 * v})) for s in (1, -1))
        assert abs((up - down) / 2e-5 - (gk * v).sum()) < 1e-6 * (1 + (gk.abs() * v.abs()).sum()), k


@pytest.mark.gpu
def test_gradients_against_the_kernels_differences():
    """The backward kernels against differences of the forward kernel, in fp32.  Along a random direction with step s the
    kernel's difference is off the 64-bit one by what y and S_T are off (T (11 m + 8) + N + 24 roundings of their
    magnitudes) over s, and the 64-bit difference off the derivative by an amount that the 64-bit form gives itself."""
    B, T, D, N, s = 1, 40, 16, 8, 2.0 ** -6
    x = inputs(B, T, D, N, 1, F32, 5, "skip z dt_bias S0")
    gen = torch.Generator().manual_seed(6)
    dy, dS = torch.randn(B, T, D, generator=gen), torch.randn(1, D, N, generator=gen)
    names = ("x", "dt", "A", "b", "c", "skip", "z", "dt_bias", "S0")
    d = to_dev(x)
    g = kda.kda_sel_scan_bwd(d["x"], d["dt"], d["A"], d["b"], d["c"], dy.to(DEV), d["S0"], dS.to(DEV), **options(d, True))
    g64, mag, r = gradients64(x, dy, dS, [(0, 0, T)], True)

    def moved(k, v, sign):
        return dict(x, **{k: (x[k] + sign * s * v).to(F32)})

    for k in names:
        v = torch.sign(torch.randn(x[k].shape, generator=gen))
        v = v * x[k].abs() if k == "A" else v
        diff = diff64 = slack = 0.0
        step = [moved(k, v, sign) for sign in (1, -1)]
        for p, sign in zip(step, (1, -1)):
            e = to_dev(p)
            y, S = kda.kda_sel_scan_fwd(e["x"], e["dt"], e["A"], e["b"], e["c"], e["S0"], **options(e, True))
            diff += sign * ((y.cpu().double() * dy).sum() + (S.cpu().double() * dS).sum()).item()
            a = sequence(p, 0, 0, T, 0)
            y64, S64 = scan64(a, True)
            diff64 += sign * ((y64 * dy[0]).sum() + (S64 * dS[0]).sum()).item()
            m = scan_magnitudes(a, True)
            rr = (T * per_token(a, True) + N + 25) * 2.0 ** -24
            slack += rr * ((m["y"] * dy[0].abs()).sum() + (m["S"] * dS[0].abs()).sum()).item()
        name = "d" + k
        along = ((step[0][k].double() - step[1][k].double()) * g[name].double().cpu()).sum().item()
        along64 = ((step[0][k].double() - step[1][k].double()) * g64[name]).sum().item()
        tol = slack + abs(diff64 - along64) + r * 2.0 ** -24 * (2 * s * v.abs() * mag[name]).sum().item()
        assert abs(diff - along) <= tol, (k, diff, along, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_no_sequence(dtype):
    """Rows before the first sequence and behind the last are neither read nor written: NaN there reaches
    nothing, and the caller's output keeps what it had; where the outputs are made here they are zero."""
    D, N, lens, first, rows = 24, 16, [40, 0, 70], 3, 120
    x = inputs(1, rows, D, N, 1, dtype, 9, "skip z dt_bias S0", n=3)
    none = torch.ones(rows, dtype=torch.bool)
    none[first:first + sum(lens)] = False
    for k in ("x", "dt", "b", "c", "z"):
        x[k][0, none] = float("nan")
    d, cu = to_dev(x), cu_of(lens, first)
    sp = [(0, lo + first, hi + first) for _, lo, hi in spans(1, rows, lens)]
    args = (d["x"], d["dt"], d["A"], d["b"], d["c"])
    kept = torch.full((1, rows, D), 5.0, dtype=dtype, device=DEV)
    y, S_T = kda.kda_sel_scan_fwd(*args, d["S0"], cu_seqlens=cu, y=kept, **options(d, True))
    check_fwd(x, y.cpu(), S_T.cpu(), sp, True, dtype)
    assert (y.cpu()[0, none] == 5).all()
    y, _ = kda.kda_sel_scan_fwd(*args, d["S0"], cu_seqlens=cu, **options(d, True))
    assert not y.cpu()[0, none].any()
    dy = torch.randn(1, rows, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    dy[0, none] = float("nan")
    got = kda.kda_sel_scan_bwd(*args, dy.to(DEV), d["S0"], cu_seqlens=cu, **options(d, True))
    for k in ("dx", "ddt", "db", "dc", "dz"):
        assert not got[k].cpu()[0, none].any(), k
    check_bwd(got, x, dy, None, sp, True, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("first,lens", [(9000, [40]), (0, [0, 1]), (0, [0]), (9001, [0, 0]), (18000, [0]), (17999, [1])])
def test_many_rows_of_no_sequence(first, lens):
    """More rows than the workgroups that clear them have lanes, before, behind and on both sides of little or nothing."""
    D, N, rows = 72, 8, 18000
    d = to_dev(inputs(1, rows, D, N, 1, F32, 9, "z", n=len(lens)))
    cu, dy = cu_of(lens, first), torch.ones(1, rows, D, device=DEV)
    args = (d["x"], d["dt"], d["A"], d["b"], d["c"])
    got = kda.kda_sel_scan_bwd(*args, dy, cu_seqlens=cu, **options(d, True))
    got["y"], _ = kda.kda_sel_scan_fwd(*args, cu_seqlens=cu, **options(d, True))
    some = slice(first, first + sum(lens))
    for k in ("y", "dx", "ddt", "db", "dc", "dz"):
        t = got[k].cpu()[0]
        assert (t[some] != 0).any() == (sum(lens) > 0), k
        t[some] = 0
        assert not t.any(), k


@pytest.mark.gpu
def test_offsets_out_of_order_stay_inside():
    """Offsets that fall or leave the range: nothing behind the tensors is touched."""
    D, N, rows = 64, 16, 300
    x = inputs(1, rows, D, N, 1, F32, 2, "S0", n=4)
    d = to_dev(x)
    cu = torch.tensor([50, 10, -7, 1 << 30, 20], dtype=torch.int32, device=DEV)
    big = torch.full((3, rows, D), 2.0, device=DEV)
    S = torch.full((3, 4, D, N), 2.0, device=DEV)
    kda.kda_sel_scan_fwd(d["x"], d["dt"], d["A"], d["b"], d["c"], d["S0"], cu_seqlens=cu, y=big[1:2], S_T=S[1])
    kda.kda_sel_scan_bwd(d["x"], d["dt"], d["A"], d["b"], d["c"], big[1:2], d["S0"], cu_seqlens=cu)
    torch.cuda.synchronize()
    for t in (big[0], big[2], S[0], S[2]):
        assert (t == 2).all()


@pytest.mark.gpu
def test_state_in_place_and_cut_sequences():
    """A sequence cut into pieces, its last state written over its first, equals the tokens in two calls, and the
    whole call in a batch that is not cut."""
    T, D, N = 700, 64, 16
    x = inputs(1, T, D, N, 1, F32, 12, "skip z dt_bias S0")
    assert kda.kda_sel_scan_fwd_workspace_size(1, T, D, N, 1) > 0
    d = to_dev(x)
    S = d["S0"].clone()
    y, S_T = kda.kda_sel_scan_fwd(d["x"], d["dt"], d["A"], d["b"], d["c"], S, S_T=S, **options(d, True))
    assert S_T is S
    check_fwd(x, y.cpu(), S.cpu(), [(0, 0, T)], True, F32)
    S2, parts = d["S0"].clone(), []
    for lo, hi in ((0, 413), (413, T)):
        cut = {k: v[:, lo:hi].contiguous() if k in ("x", "dt", "b", "c", "z") else v for k, v in d.items()}
        yp, S2 = kda.kda_sel_scan_fwd(cut["x"], cut["dt"], cut["A"], cut["b"], cut["c"], S2, **options(cut, True))
        parts.append(yp)
    check_fwd(x, torch.cat(parts, 1).cpu(), S2.cpu(), [(0, 0, T)], True, F32)


def decode(x, slots, ntok, T, y=None, softplus=True):
    d = to_dev(x)
    t = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)   # noqa: E731
    y = kda.kda_sel_scan_step(d["x"], d["dt"], d["A"], d["b"], d["c"], d["S0"], slots=t(slots), ntok=t(ntok), y=None if y is None else y.to(DEV),
                              **options(d, softplus))
    torch.cuda.synchronize()
    return y.cpu(), d["S0"].cpu()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,D,N,G,parts,softplus", [(1, 1, 8, 8, 1, "S0", False), (3, 1, 72, 16, 1, "skip z dt_bias S0", True),
                                                      (2, 5, 136, 32, 1, "skip z dt_bias S0", True), (2, 9, 48, 64, 2, "z S0", True)])
def test_step(B, T, D, N, G, parts, softplus, dtype):
    print(f"scan step B={B} T={T} D={D} N={N} G={G} {parts} {dtype}", flush=True)
    x = inputs(B, T, D, N, G, dtype, 6, parts, softplus)
    y, S = decode(x, None, None, T, softplus=softplus)
    check_fwd(x, y, S, spans(B, T, None), softplus, dtype)


@pytest.mark.gpu
def test_step_slots_padding_and_duplicates():
    """As kda_gdr_step: a pool larger than the batch, rows padded by slot, by length, and by a slot that an
    earlier row with tokens has; what is padded keeps its y, what no row names its state."""
    B, T, D, N, P = 9, 3, 40, 16, 12
    x = inputs(B, T, D, N, 1, BF16, 3, "skip z dt_bias S0", n=P)
    slots = [5, -1, 0, 11, 5, 12, 7, 2, 1 << 30]
    ntok = [0, 3, 1, 9, 3, 2, 0, 2, 1]
    real = {2: 1, 3: 3, 4: 3, 7: 2}
    y0 = torch.full((B, T, D), 7.0).to(BF16)
    y, S = decode(x, slots, ntok, T, y0)
    for b, n in real.items():
        a = sequence(x, b, 0, n, slots[b])
        y64, S64 = scan64(a, True)
        m, r = scan_magnitudes(a, True), n * per_token(a, True) + N + 24
        close(y[b, :n], y64, BF16, m["y"], r, f"y of row {b}")
        close(S[slots[b]], S64, F32, m["S"], r, f"state {slots[b]}")
        assert torch.equal(y[b, n:], y0[b, n:])
    for b in set(range(B)) - set(real):
        assert torch.equal(y[b], y0[b]), b
    for s in set(range(P)) - {slots[b] for b in real}:
        assert torch.equal(S[s], x["S0"][s]), s


@pytest.mark.gpu
def test_not_finite_stays_in_its_place():
    """NaN in one channel's x stays in that channel behind its token, an infinity in b in its group, and nothing reaches other
    sequences; a step size of infinity forgets the state, one of zero keeps it."""
    T, D, N = 70, 32, 16
    x = inputs(3, T, D, N, 2, F32, 7, "skip S0", softplus=False)
    x["x"][0, 20, 3] = float("nan")
    x["b"][1, 30, 1, 2] = float("inf")
    x["dt"][2, 10, 5] = float("inf")
    x["x"][2, 10, 5] = 0.0
    x["dt"][2, :, 6] = 0.0
    d = to_dev(x)
    y, S = kda.kda_sel_scan_fwd(d["x"], d["dt"], d["A"], d["b"], d["c"], d["S0"], **options(d, False))
    y, S = y.cpu(), S.cpu()
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 20:, 3] = True
    want[1, 30:, 16:] = True
    want[2, 10:, 5] = True   # infinity times zero
    assert torch.equal(bad, want)
    assert torch.equal(S[2, 6], x["S0"][2, 6])


@pytest.mark.gpu
def test_graph_other_stream_and_repeats():
    """A captured call, replayed with other inputs and eager work between, equals the eager one bit for bit; so do calls
    on another stream, with a workspace of the caller's."""
    T, D, N = 300, 64, 16
    x = [to_dev(inputs(1, T, D, N, 1, BF16, s, "skip z dt_bias S0")) for s in (1, 2)]
    st = {k: None if v is None else v.clone() for k, v in x[0].items()}
    dy = torch.randn(1, T, D, device=DEV).to(BF16)

    def call(a, **kw):
        y, S = kda.kda_sel_scan_fwd(a["x"], a["dt"], a["A"], a["b"], a["c"], a["S0"], **options(a, True), **kw.get("f", {}))
        g = kda.kda_sel_scan_bwd(a["x"], a["dt"], a["A"], a["b"], a["c"], dy, a["S0"], **options(a, True), **kw.get("b", {}))
        return [y, S] + [g[n] for n in NAMES]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(st)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(st)
    for i in (0, 1, 0, 1):
        for k, v in st.items():
            v.copy_(x[i][k])
        graph.replay()
        torch.cuda.synchronize()
        want = call(x[i])
        for a, b in zip(out, want):
            assert torch.equal(a, b)
    ws = dict(f=dict(stream=side, workspace=torch.empty(kda.kda_sel_scan_fwd_workspace_size(1, T, D, N, 1) + 64, dtype=torch.uint8, device=DEV)),
              b=dict(stream=side, workspace=torch.empty(kda.kda_sel_scan_bwd_workspace_size(1, T, D, N, 1) + 64, dtype=torch.uint8, device=DEV)))
    torch.cuda.synchronize()
    got = call(x[1], **ws)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ----------------------------------------------------------------------------- refusals (no GPU)
class Fake:
    """Disjoint addresses that are never read."""

    def __init__(self, **over):
        self.v = dict(dtype=0, n=2, T=64, D=64, N=16, G=1, softplus=1)
        self.ptr = {k: (1 << 40) + (i << 30) for i, k in enumerate(
            "cu x dt A b c skip z dt_bias S0 dy dS_T y S_T ws dx ddt dA db dc dskip dz ddt_bias dS0 slots ntok".split())}
        self.ptr["cu"] = None
        self.ws, self.rest = 1 << 29, 1
        self.nslot = 4
        for k, v in over.items():
            if k in self.v:
                self.v[k] = v
            elif k in self.ptr:
                self.ptr[k] = v
            else:
                setattr(self, k, v)

    def p(self, *names):
        return [None if self.ptr[n] is None else ctypes.c_void_p(self.ptr[n]) for n in names]

    def sizes(self):
        return [self.v[k] for k in ("dtype", "n", "T", "D", "N", "G", "softplus")]

    IN = ("cu", "x", "dt", "A", "b", "c", "skip", "z", "dt_bias", "S0")

    def fwd(self, lib):
        return lib.kda_sel_scan_fwd(*self.sizes(), *self.p("cu"), self.rest, *self.p(*self.IN[1:], "y", "S_T", "ws"), self.ws, None)

    def bwd(self, lib):
        return lib.kda_sel_scan_bwd(*self.sizes(), *self.p(*self.IN, "dy", "dS_T", "dx", "ddt", "dA", "db", "dc", "dskip", "dz", "ddt_bias", "dS0", "ws"),
                                    self.ws, None)

    def step(self, lib):
        s = self.sizes()
        return lib.kda_sel_scan_step(*s[:6], self.nslot, s[6], *self.p("x", "dt", "A", "b", "c", "skip", "z", "dt_bias", "S0", "slots", "ntok", "y"), None)


@pytest.fixture(scope="module")
def lib():
    try:
        return kda.load_library()
    except RuntimeError as e:
        pytest.skip(str(e))


NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, ALIAS = 1, 2, 3, 4, 5, 6


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), DTYPE), (dict(n=0), SHAPE), (dict(T=0), SHAPE), (dict(T=(1 << 30) + 1), SHAPE), (dict(D=60), SHAPE), (dict(D=0), SHAPE),
    (dict(D=1 << 21), SHAPE), (dict(G=0), SHAPE), (dict(G=3), SHAPE), (dict(G=16), SHAPE), (dict(N=12), SHAPE), (dict(N=128), SHAPE),
    (dict(softplus=2), SHAPE), (dict(n=1 << 26), SHAPE), (dict(x=None), NULL), (dict(A=None), NULL), (dict(c=None), NULL), (dict(dt=(1 << 40) + 4), ALIGN),
    (dict(skip=(1 << 41) + 8), ALIGN)])
def test_refusals_of_all(lib, over, status):
    for call in ("fwd", "bwd", "step"):
        assert getattr(Fake(**over), call)(lib) == status, call


def test_refusals_of_each(lib):
    at = Fake().ptr
    assert Fake(rest=2).fwd(lib) == SHAPE and Fake(rest=-1).fwd(lib) == SHAPE
    assert Fake(y=None).fwd(lib) == NULL and Fake(dA=None).bwd(lib) == NULL and Fake(y=None).step(lib) == NULL
    assert Fake(y=at["x"]).fwd(lib) == ALIAS and Fake(S_T=at["x"]).fwd(lib) == ALIAS and Fake(y=at["S_T"]).fwd(lib) == ALIAS
    assert Fake(S_T=at["S0"] + 16).fwd(lib) == ALIAS
    assert Fake(ws=None).bwd(lib) == WORKSPACE
    assert Fake(z=None).bwd(lib) == NULL and Fake(dz=None).bwd(lib) == NULL and Fake(skip=None).bwd(lib) == NULL and Fake(dt_bias=None).bwd(lib) == NULL
    assert Fake(dx=at["dy"]).bwd(lib) == ALIAS and Fake(db=at["dc"]).bwd(lib) == ALIAS and Fake(dS0=at["S0"]).bwd(lib) == ALIAS
    assert Fake(nslot=0).step(lib) == SHAPE and Fake(nslot=1, slots=None).step(lib) == SHAPE
    assert Fake(y=at["S0"]).step(lib) == ALIAS and Fake(S0=at["slots"]).step(lib) == ALIAS
    small = Fake()
    small.ws = 8
    assert small.bwd(lib) == WORKSPACE


def test_workspace_sizes(lib):
    size = ctypes.c_size_t(0)
    for name in ("kda_sel_scan_fwd_workspace_size", "kda_sel_scan_bwd_workspace_size"):
        fn = getattr(lib, name)
        assert fn(1, 64, 64, 16, 1, 0, None) == NULL
        assert fn(1, 64, 64, 12, 1, 0, ctypes.byref(size)) == SHAPE
        last = 0
        for T in (64, 4096, 65536):
            assert fn(1, T, 64, 16, 1, 1, ctypes.byref(size)) == 0
            assert size.value >= last
            last = size.value
    # a long sequence of few channels is cut, a batch that fills the device is not
    assert kda.kda_sel_scan_fwd_workspace_size(1, 65536, 64, 16, 1) > 0
    assert kda.kda_sel_scan_fwd_workspace_size(64, 4096, 4096, 16, 1) == 0


def test_binding_refuses(lib):
    x = inputs(1, 4, 8, 8, 1, F32, 0)
    call = lambda **o: kda.kda_sel_scan_fwd(*[dict(x, **o)[k] for k in ("x", "dt", "A", "b", "c")])   # noqa: E731
    with pytest.raises(ValueError):   # on the CPU
        call()
    with pytest.raises(TypeError):
        call(dt=x["dt"].double())
    with pytest.raises(ValueError):
        call(b=x["b"][:, :2])
    with pytest.raises(ValueError):
        call(x=x["x"].transpose(0, 1).expand(4, 2, 8)[:, :1].transpose(0, 1))
    with pytest.raises(TypeError):
        call(x=x["x"].half(), dt=x["dt"].half(), b=x["b"].half(), c=x["c"].half())
