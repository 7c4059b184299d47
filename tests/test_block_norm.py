"""kda_block_norm_fwd and kda_block_norm_bwd against the definition in 64 bits.

Tolerances count fp32 roundings: a mean of squares over D is a chain of 8 additions in a
lane and log2 of the lanes beyond it (at most 10 + 8 further), its reciprocal root and the
products that follow are a few more, so a row's values carry at most ~40 roundings of the
magnitudes they are made of; a hardware exponential's argument is rounded once, which at
|z| <= 12 is worth 12 more.  64 covers them.  Backward values pass through two such norms:
160.  Weight gradients add one rounding a row.  Each stored result is rounded once more.
"""
import ctypes
import itertools

import pytest
import torch

import chunked_gated_delta_12_amd as kda
from plain_ops import U32, close, norm64

DEV = "cuda:0"
NAMES = ("x", "y", "z", "w_post", "s", "w_pre")
EPS = 1e-6


def make(lead, D, dtype, seed, parts):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    a = dict(y=(0.7 * n(*lead, D)).to(dtype), x=(2 * n(*lead, D)).to(dtype), z=(2 * n(*lead, D)).to(dtype),
             w_post=1 + 0.1 * n(D), s=0.3 + 0.1 * n(D), w_pre=1 + 0.1 * n(D))
    a = {k: v if k == "y" or k in parts else None for k, v in a.items()}
    a["dr"], a["dh"] = n(*lead, D).to(dtype), n(*lead, D).to(dtype) if "w_pre" in parts else None
    return a


def gpu(a):
    return {k: None if v is None else v.to(DEV) for k, v in a.items()}


def check(lead, D, dtype, seed, parts, act, eps=EPS, use_dr=True, **kw):
    a = make(lead, D, dtype, seed, parts)
    if not use_dr:
        a["dr"] = None
    d = gpu(a)
    print(f"norm lead={lead} D={D} {dtype} {sorted(parts)} {act}", flush=True)
    opt = {k: d[k] for k in NAMES if k != "y"}
    r, h = kda.kda_block_norm_fwd(d["y"], act=act, eps=eps, **opt, **kw)
    g = kda.kda_block_norm_bwd(d["y"], d["dr"], d["dh"], act=act, eps=eps, **opt)
    torch.cuda.synchronize()
    b = {k: None if a[k] is None else a[k].double().requires_grad_() for k in NAMES}
    r64, h64 = norm64(b, act, eps)
    rms = lambda t: 1 / torch.sqrt(t.detach().pow(2).mean(-1, keepdim=True) + eps)   # noqa: E731
    part = r64.detach() if a["x"] is None else (r64 - b["x"]).detach()
    mag_r = part.abs() + (0 if a["x"] is None else b["x"].detach().abs())
    close(r, r64, dtype, mag_r, 64, "r")
    if h64 is not None:
        # h = r rho w: r's error and rho's
        mag_h = (mag_r + r64.detach().abs()) * rms(r64) * b["w_pre"].detach().abs() + h64.detach().abs() * (mag_r * rms(r64)).pow(2).mean(-1, keepdim=True).sqrt()
        close(h, h64, dtype, mag_h, 64, "h")
    loss = 0
    if a["dr"] is not None:
        loss = loss + (r64 * a["dr"].double()).sum()
    if a["dh"] is not None:
        loss = loss + (h64 * a["dh"].double()).sum()
    have = [k for k in NAMES if a[k] is not None]
    ref = dict(zip(have, torch.autograd.grad(loss, [b[k] for k in have], allow_unused=True)))
    nrow = a["y"].numel() // D
    for k in NAMES:
        if a[k] is None:
            assert g["d" + k] is None
            continue
        want = ref[k] if ref[k] is not None else torch.zeros_like(b[k])
        if k in ("x", "y", "z"):
            # magnitudes: a row's gradients are differences of terms of the row's largest size
            mag = want.abs() + 4 * grad_scale(a, b, k, act, eps)
            close(g["d" + k], want, dtype, mag, 160, "d" + k)
        else:
            # sums over rows, then the same number of roundings as a value
            tot = weight_scale(a, b, k, act, eps)
            close(g["d" + k], want, torch.float32, tot, 160 + nrow, "d" + k)
    return r, h, g


def _sizes(a, b, act, eps):
    """Per element: |dr'| bound, |n|, |act|, |act'| (float64)."""
    rms = lambda t: 1 / torch.sqrt(t.pow(2).mean(-1, keepdim=True) + eps)   # noqa: E731
    with torch.no_grad():
        y = b["y"]
        n = (y * rms(y) * b["w_post"] if b["w_post"] is not None else y).abs()
        al, sl = torch.ones_like(y), torch.ones_like(y)
        if b["z"] is not None:
            sg = torch.sigmoid(b["z"])
            al = (b["z"].abs() if act == "silu" else 1) * sg
            sl = sg * (1 + b["z"].abs()) if act == "silu" else sg
        dr = a["dr"].double().abs() if a["dr"] is not None else torch.zeros_like(y)
        if a["dh"] is not None:
            r = norm64(b, act, eps)[0]
            t = (a["dh"].double() * b["w_pre"]).abs()
            big = r.abs() if b["x"] is None else r.abs() + b["x"].abs() + (r - b["x"]).abs()
            dr = dr + rms(r) * t * 2 + big * rms(r) ** 3 * (t * big).mean(-1, keepdim=True) * 3
        return dr, n, al, sl, rms(y)


def grad_scale(a, b, k, act, eps):
    dr, n, al, sl, ry = _sizes(a, b, act, eps)
    s = b["s"].detach().abs() if b["s"] is not None else 1.0
    if k == "x":
        return dr
    if k == "z":
        return dr * s * n * sl
    dn = dr * s * al
    if b["w_post"] is None:
        return dn
    c = dn * b["w_post"].detach().abs()
    y = b["y"].detach().abs()
    return ry * c + y * ry ** 3 * (c * y).mean(-1, keepdim=True)


def weight_scale(a, b, k, act, eps):
    dr, n, al, sl, ry = _sizes(a, b, act, eps)
    s = b["s"].detach().abs() if b["s"] is not None else 1.0
    if k == "s":
        t = dr * n * al
    elif k == "w_post":
        t = dr * s * al * b["y"].detach().abs() * ry
    else:
        with torch.no_grad():
            r = norm64(b, act, eps)[0]
            rr = 1 / torch.sqrt(r.pow(2).mean(-1, keepdim=True) + eps)
            big = r.abs() if b["x"] is None else r.abs() + b["x"].abs() + (r - b["x"]).abs()
            t = a["dh"].double().abs() * big * rr * 3
    return t.reshape(-1, t.shape[-1]).sum(0)


ALL = ("x", "z", "w_post", "s", "w_pre")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [8, 16, 24, 40, 64, 128, 136, 512, 520, 1000, 1024, 2048, 2056, 4104, 8192])
def test_every_width(D, dtype):
    check((13,), D, dtype, D, ALL, "silu" if D % 16 else "sigmoid")


@pytest.mark.gpu
@pytest.mark.parametrize("parts", [c for n in range(6) for c in itertools.combinations(ALL, n)])
def test_every_set_of_parts(parts):
    check((5, 7), 64, torch.float32, 3, parts, "silu")
    check((9,), 520, torch.bfloat16, 4, parts, "sigmoid")


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 2, 3, 16, 17, 4099, 70001])
def test_rows(rows):
    check((rows,), 64, torch.bfloat16, rows, ("z", "w_post"), "silu")
    if rows < 5000:
        check((rows,), 1000, torch.float32, rows, ALL, "sigmoid")


@pytest.mark.gpu
def test_without_dr():
    check((12,), 256, torch.float32, 1, ALL, "sigmoid", use_dr=False)


@pytest.mark.gpu
def test_residual_in_place():
    a = gpu(make((33,), 256, torch.bfloat16, 5, ALL))
    opt = {k: a[k] for k in ("z", "w_post", "s", "w_pre")}
    r, h = kda.kda_block_norm_fwd(a["y"], x=a["x"], **opt)
    x = a["x"].clone()
    r2, h2 = kda.kda_block_norm_fwd(a["y"], x=x, r=x, **opt)
    assert r2 is x and torch.equal(r, x) and torch.equal(h, h2)


@pytest.mark.gpu
def test_extreme_rows():
    """A row of zeros (eps alone under the root), one of large values, gates far out."""
    y = torch.zeros(4, 64)
    y[1] = 1e15
    y[2] = 1e-15
    y[3] = 1.0
    z = torch.tensor([-200.0, 200.0, 0.0, -80.0])[:, None].expand(4, 64).contiguous()
    w = torch.ones(64)
    for act in ("sigmoid", "silu"):
        r, h = kda.kda_block_norm_fwd(y.to(DEV), z=z.to(DEV), w_post=w.to(DEV), w_pre=w.to(DEV), act=act)
        r64, h64 = norm64(dict(y=y.double(), x=None, z=z.double(), w_post=w.double(), s=None, w_pre=w.double()), act, EPS)
        assert torch.isfinite(r).all() and torch.isfinite(h).all()
        # e^-80's argument is rounded at 80: 80 roundings more; what is below fp32's range is zero
        close(r, r64, torch.float32, r64.abs() + 2.0 ** -126 / U32, 160, "r")


@pytest.mark.gpu
def test_nan_stays_in_its_row():
    a = gpu(make((40,), 64, torch.bfloat16, 6, ALL))
    opt = {k: a[k] for k in ("x", "z", "w_post", "s", "w_pre")}
    r, h = kda.kda_block_norm_fwd(a["y"], **opt)
    d = kda.kda_block_norm_bwd(a["y"], a["dr"], a["dh"], **opt)
    a["y"][17, 3] = float("nan")
    r2, h2 = kda.kda_block_norm_fwd(a["y"], **opt)
    d2 = kda.kda_block_norm_bwd(a["y"], a["dr"], a["dh"], **opt)
    keep = torch.arange(40, device=DEV) != 17
    for one, two in ((r, r2), (h, h2), (d["dx"], d2["dx"]), (d["dy"], d2["dy"]), (d["dz"], d2["dz"])):
        assert torch.equal(one[keep], two[keep]) and two[17].isnan().any()
    assert d2["dw_pre"].isnan().all() and d2["dw_post"].isnan().any()


@pytest.mark.gpu
def test_repeats_bit_for_bit_and_on_a_stream():
    a = gpu(make((3001,), 136, torch.bfloat16, 7, ALL))
    opt = {k: a[k] for k in ("x", "z", "w_post", "s", "w_pre")}
    one = kda.kda_block_norm_bwd(a["y"], a["dr"], a["dh"], **opt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    two = kda.kda_block_norm_bwd(a["y"], a["dr"], a["dh"], stream=side, **opt)
    torch.cuda.current_stream().wait_stream(side)
    for k in one:
        assert torch.equal(one[k], two[k]), k


@pytest.mark.gpu
def test_captured():
    """Forward and backward in a graph, replayed on new inputs between eager calls."""
    a = gpu(make((65,), 1000, torch.bfloat16, 8, ALL))
    opt = {k: a[k] for k in ("x", "z", "w_post", "s", "w_pre")}
    kda.kda_block_norm_bwd(a["y"], a["dr"], a["dh"], **opt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, h = kda.kda_block_norm_fwd(a["y"], **opt)
        d = kda.kda_block_norm_bwd(a["y"], a["dr"], a["dh"], **opt)
    for i in range(4):
        a["y"].copy_(torch.randn(65, 1000, generator=torch.Generator().manual_seed(i)).to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        r2, h2 = kda.kda_block_norm_fwd(a["y"], **opt)
        d2 = kda.kda_block_norm_bwd(a["y"], a["dr"], a["dh"], **opt)
        torch.cuda.synchronize()
        assert torch.equal(r, r2) and torch.equal(h, h2)
        for k in d:
            assert torch.equal(d[k], d2[k]), (i, k)


@pytest.mark.gpu
def test_gradients_by_differences():
    """Central differences of the kernel's own forward in fp32: the loss moves by 2 eps <grad, v>."""
    a = gpu(make((6,), 64, torch.float32, 9, ALL))
    opt = {k: a[k] for k in ("x", "z", "w_post", "s", "w_pre")}
    d = kda.kda_block_norm_bwd(a["y"], a["dr"], a["dh"], act="silu", **opt)

    def loss(b):
        r, h = kda.kda_block_norm_fwd(b["y"], act="silu", **{k: b[k] for k in opt})
        return float((r.double() * a["dr"].double()).sum() + (h.double() * a["dh"].double()).sum())

    gen = torch.Generator().manual_seed(1)
    step = 2.0 ** -8   # the truncation is of the order step^2 = 2^-16, the roundings 2^-24 / step = 2^-16
    for k in NAMES:
        v = torch.randn(a[k].shape, generator=gen).to(DEV)
        v = v / v.norm()
        up, down = (loss({**a, k: a[k] + sgn * step * v}) for sgn in (1, -1))
        want = float((d["d" + k].double() * v.double()).sum())
        assert abs((up - down) / (2 * step) - want) <= 2.0 ** -9 * float(d["d" + k].double().norm()), k


# ----------------------------------------------------------------------------- refusals (no GPU)
@pytest.fixture(scope="module")
def lib():
    try:
        return kda.load_library()
    except RuntimeError as e:
        pytest.skip(str(e))


def _addr(names, n):
    base, out = 1 << 40, {}
    for name in names:
        out[name] = base
        base += n + 4096
    return out


def test_forward_refusals(lib):
    a = _addr(("y", "x", "z", "w_post", "s", "w_pre", "r", "h"), 1 << 16)

    def call(dtype=0, act=0, rows=8, D=64, eps=1e-6, **over):
        b = {**a, **over}
        p = [None if b[k] is None else ctypes.c_void_p(b[k]) for k in ("y", "x", "z", "w_post", "s", "w_pre", "r", "h")]
        return lib.kda_block_norm_fwd(dtype, act, rows, D, eps, *p, None)

    assert call(dtype=2) == 3 and call(act=2) == 2
    assert call(rows=0) == 2 and call(rows=1 << 50) == 2
    for D in (0, 4, 12, 8200, 1 << 30):
        assert call(D=D) == 2, D
    assert call(eps=-1e-3) == 2 and call(eps=float("nan")) == 2 and call(eps=2.0) == 2
    assert call(y=None) == 1 and call(r=None) == 1 and call(h=None) == 1 and call(w_pre=None) == 1
    assert call(z=a["z"] + 8) == 4 and call(s=a["s"] + 4) == 4
    assert call(r=a["y"]) == 6 and call(r=a["z"]) == 6 and call(r=a["x"] + 16) == 6
    assert call(h=a["r"]) == 6 and call(h=a["x"]) == 6 and call(h=a["w_pre"]) == 6


def test_backward_refusals(lib):
    order = ("y", "x", "z", "w_post", "s", "w_pre", "dr", "dh", "dy", "dx", "dz", "dw_post", "ds", "dw_pre", "ws")
    a = _addr(order, 1 << 20)
    need = kda.kda_block_norm_bwd_workspace_size(8, 64)
    assert need > 0

    def call(ws_bytes=1 << 20, **over):
        b = {**a, **over}
        return lib.kda_block_norm_bwd(0, 0, 8, 64, 1e-6, *[None if b[k] is None else ctypes.c_void_p(b[k]) for k in order],
                                      ws_bytes, None)

    assert call(y=None) == 1 and call(dy=None) == 1 and call(dh=None) == 1 and call(w_pre=None) == 1
    assert call(dr=None, dh=None, w_pre=None, dw_pre=None) == 1
    assert call(x=None) == 1 and call(z=None) == 1 and call(s=None) == 1   # a gradient of what is not there
    assert call(ws_bytes=need - 1) == 5 and call(ws=None) == 5
    assert call(dx=a["dr"]) == 6 and call(dy=a["y"]) == 6 and call(dz=a["dy"]) == 6 and call(dw_pre=a["ws"]) == 6
    assert call(dy=a["dy"] + 2) == 4
    with pytest.raises(kda.KdaError):
        kda.kda_block_norm_bwd_workspace_size(0, 64)


def test_binding_refusals(lib):
    y = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        kda.kda_block_norm_fwd(y, act="relu")
    with pytest.raises(TypeError):
        kda.kda_block_norm_fwd(y.half())
    with pytest.raises(ValueError):
        kda.kda_block_norm_fwd(y, x=torch.zeros(4, 32))
    with pytest.raises(TypeError):
        kda.kda_block_norm_fwd(y, w_post=torch.ones(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        kda.kda_block_norm_fwd(torch.zeros(64, 4).t())   # not contiguous
    with pytest.raises(ValueError):
        kda.kda_block_norm_fwd(y)                        # not on the GPU


def test_workspace_of_the_caller_is_checked(lib):
    y, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError, match="workspace is on"):
        kda.kda_block_norm_bwd(y, y, w_post=w, workspace=torch.empty(1 << 20, dtype=torch.uint8, device="meta"))
    with pytest.raises(TypeError, match="workspace"):
        kda.kda_block_norm_bwd(y, y, w_post=w, workspace=b"")


@pytest.mark.gpu
def test_two_calls_at_once():
    """Two streams, each call with a workspace of its own: what each gives alone, bit for bit."""
    ds = [gpu(make((3000,), 1000, torch.bfloat16, 60 + i, {"x", "z", "w_post", "s", "w_pre"})) for i in range(2)]

    def call(d, stream):
        opt = {k: d[k] for k in NAMES if k != "y"}
        g = kda.kda_block_norm_bwd(d["y"], d["dr"], d["dh"], stream=stream, **opt)
        return [*kda.kda_block_norm_fwd(d["y"], stream=stream, **opt)] + [g[k] for k in sorted(g)]

    want = []
    for d in ds:
        want.append(call(d, None))
        torch.cuda.synchronize()
    got = [call(d, s) for d, s in zip(ds, [torch.cuda.Stream() for _ in ds])]
    torch.cuda.synchronize()
    for p, q in zip(want, got):
        for j, (u, v) in enumerate(zip(p, q)):
            assert torch.equal(u, v), j


@pytest.mark.gpu
@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-30])
@pytest.mark.parametrize("rows,D,dtype", [(17, 8, torch.float32), (17, 128, torch.bfloat16), (5, 64, torch.float32), (2049, 1000, torch.bfloat16),
                                          (3, 1000, torch.float32), (1, 24, torch.bfloat16), (3, 2048, torch.bfloat16)])
def test_eps_of_zero_and_part_groups(rows, D, dtype, eps):
    """Rows that do not fill the last group of lanes: where no row is, the root of zero stands under nothing,
    and the weights' gradients are those of the rows."""
    check((rows,), D, dtype, 100 + rows + D, ALL, "silu", eps=eps)
    check((rows,), D, dtype, 101 + rows + D, ("w_pre",), "sigmoid", eps=eps)
    check((rows,), D, dtype, 102 + rows + D, ("z", "w_post"), "sigmoid", eps=eps)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 1000, 8192])
@pytest.mark.parametrize("power", [-50, -43, 43, 50])
def test_rows_of_any_scale(power, D):
    """With eps 0 the norms do not see a row's scale.  Scaled by a power of two every step scales with it
    exactly, while it stays in range: the same bits, times the power or over it."""
    by = 2.0 ** power
    a = gpu(make((7,), D, torch.float32, 120 + D, ("z", "s", "w_post", "w_pre")))
    kw = dict(z=a["z"], s=a["s"], act="silu", eps=0.0)
    # the norm after the block: r is the same, y's gradient over the scale
    one, two = (kda.kda_block_norm_bwd(y, a["dr"], w_post=a["w_post"], **kw) for y in (a["y"], a["y"] * by))
    assert torch.equal(one["dy"], two["dy"] * by)
    for k in ("dz", "ds", "dw_post"):
        assert torch.equal(one[k], two[k]), k
    # the norm before the next one alone
    h1, h2 = (kda.kda_block_norm_fwd(y, w_pre=a["w_pre"], **kw)[1] for y in (a["y"], a["y"] * by))
    one, two = (kda.kda_block_norm_bwd(y, None, a["dh"], w_pre=a["w_pre"], **kw) for y in (a["y"], a["y"] * by))
    assert torch.equal(h1, h2) and torch.equal(one["dy"], two["dy"] * by)
    for k in ("dz", "ds", "dw_pre"):
        assert torch.equal(one[k], two[k]), k
