"""kda_layer_norm_fwd and _bwd against the definition in 64 bits.

Tolerance, in fp32 roundings (2^-24).  A sum over D channels is one of 8 in a lane, up to 6 across
lanes and up to 16 across wavefronts: s = 32 roundings of the sum of sizes.  r has one.  With M the largest |r| of a
row, u' = r - mean is off by (s + 3) M; its squares' mean, and with it rho = 1 / sqrt(var + eps), relatively by
2 (s + 3) M / std + s + 8 (std with eps in it), half of which goes to rho; so u = u' rho by (s + 3) M / std + |u| times that, and h by |w| times it
and 3 more roundings of what is added.  Backwards, with E that bound of u over a row and t = dh w, T the mean of |t| and Q = mean |t u|:
dy is off by rho times (the relative error of rho times the three terms' sizes, E (Q + |u| T) for u, and s + 6 roundings of the terms), dw by sum |dh| E and db by the
sum's roundings (rows of a workgroup one after another, then 32: at most rows + 32).
"""
import ctypes

import pytest
import torch

import chunked_gated_delta_12_amd as kda
from plain_ops import U32, close
from plain_state_space import layer_norm64

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
SUM = 32


def inputs(rows, D, dtype, seed, parts, offset=0.3):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    a = dict(y=(0.7 * r(rows, D) + offset).to(dtype), x=(2 * r(rows, D)).to(dtype) if "x" in parts else None,
             w=1 + 0.1 * r(D) if "w" in parts else None, b=0.1 * r(D) if "b" in parts else None)
    g = dict(dh=r(rows, D).to(dtype), dr=r(rows, D).to(dtype) if "x" in parts else None)
    return a, g


def to_dev(x):
    return {k: None if v is None else v.to(DEV) for k, v in x.items()}


def f64(a):
    return {k: None if v is None else v.double() for k, v in a.items()}


def bounds(a, eps):
    """(u, rho, relative error of rho, error of u) of every row in units of one rounding."""
    r = a["y"] if a["x"] is None else a["x"] + a["y"]
    size = a["y"].abs() if a["x"] is None else a["x"].abs() + a["y"].abs()
    M = size.max(-1, keepdim=True).values
    u = r - r.mean(-1, keepdim=True)
    rho = 1 / torch.sqrt(u.pow(2).mean(-1, keepdim=True) + eps)
    rel = ((SUM + 3) * M * rho * 2 + SUM + 8) / 2 + 2
    u = u * rho
    return u, rho, rel, (SUM + 3) * M * rho + u.abs() * rel


def check_fwd(a, r, h, eps, dtype):
    a = f64(a)
    r64, h64 = layer_norm64(a, eps)
    if a["x"] is None:
        assert r is None
    else:
        close(r, r64, dtype, a["x"].abs() + a["y"].abs(), 1, "r")
    u, _, _, E = bounds(a, eps)
    w = 1.0 if a["w"] is None else a["w"].abs()
    mag = E * w + 3 * (u.abs() * w + (0.0 if a["b"] is None else a["b"].abs()))
    close(h, h64, dtype, mag, 1, "h")


def check_bwd(got, a, g, eps, dtype):
    a, g = f64(a), f64(g)
    leaves = {k: a[k].requires_grad_() for k in ("y", "w", "b") if a[k] is not None}
    r, h = layer_norm64(a, eps)
    loss = (h * g["dh"]).sum() + (0 if g["dr"] is None else (r * g["dr"]).sum())
    want = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    a = {k: None if v is None else v.detach() for k, v in a.items()}
    u, rho, rel, E = bounds(a, eps)
    t = g["dh"] if a["w"] is None else g["dh"] * a["w"]
    T, Q = t.abs().mean(-1, keepdim=True), (t * u).abs().mean(-1, keepdim=True)
    terms = t.abs() + T + u.abs() * Q
    e = rho * ((rel + SUM + 6) * terms + E * Q + u.abs() * (t.abs() * E).mean(-1, keepdim=True))
    close(got["dy"], want["y"], dtype, e + (0.0 if g["dr"] is None else 2 * g["dr"].abs()), 1, "dy")
    n = u.shape[0] + 32
    if a["w"] is not None:
        close(got["dw"], want["w"], F32, (g["dh"].abs() * E).sum(0) + n * (g["dh"] * u).abs().sum(0), 1, "dw")
    else:
        assert got["dw"] is None
    if a["b"] is not None:
        close(got["db"], want["b"], F32, n * g["dh"].abs().sum(0), 1, "db")


def both(a, g, eps, dtype, **kw):
    d, e = to_dev(a), to_dev(g)
    r, h = kda.kda_layer_norm_fwd(d["y"], x=d["x"], w=d["w"], b=d["b"], eps=eps)
    got = kda.kda_layer_norm_bwd(d["y"], e["dh"], e["dr"], x=d["x"], w=d["w"], want_db=d["b"] is not None, eps=eps)
    torch.cuda.synchronize()
    cpu = lambda t: None if t is None else t.cpu()   # noqa: E731
    return cpu(r), cpu(h), {k: cpu(v) for k, v in got.items()}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,D,parts", [(1, 8, "xwb"), (3, 16, "w"), (7, 24, "b"), (130, 64, "xwb"), (65, 136, "x"), (33, 264, "xw"), (17, 520, "xwb"),
                                          (9, 1000, "wb"), (5, 2056, "xwb"), (3, 4104, "xb"), (4, 8192, "xwb"), (3000, 32, "xwb"), (1500, 1032, "xwb"), (5, 1536, "xw"),
                                          (900, 2560, "xwb"), (4, 2568, "xb"), (3, 3584, "wb"), (4, 4096, "xwb"), (450, 5120, "xwb"), (3, 5128, "xwb"),
                                          (2, 6152, "xwb"), (3, 7168, "xwb"), (2, 7176, "x")])
def test_fwd_and_bwd(rows, D, parts, dtype):
    print(f"layer norm rows={rows} D={D} {parts} {dtype}", flush=True)
    a, g = inputs(rows, D, dtype, 3, parts)
    r, h, got = both(a, g, 1e-5, dtype)
    check_fwd(a, r, h, 1e-5, dtype)
    check_bwd(got, a, g, 1e-5, dtype)


@pytest.mark.gpu
def test_rows_far_from_zero():
    """Rows whose mean is a thousand times their spread: the squares are of r less its mean."""
    a, g = inputs(20, 512, F32, 5, "wb", offset=700.0)
    r, h, got = both(a, g, 1e-5, F32)
    check_fwd(a, r, h, 1e-5, F32)
    check_bwd(got, a, g, 1e-5, F32)


def test_plain_gradients_against_differences():
    gen = torch.Generator().manual_seed(0)
    y, x, w, b = (torch.randn(*s, generator=gen).double().requires_grad_() for s in ((3, 8), (3, 8), (8,), (8,)))
    assert torch.autograd.gradcheck(lambda y, x, w, b: layer_norm64(dict(y=y, x=x, w=w, b=b), 1e-5), (y, x, w, b))


@pytest.mark.gpu
def test_equal_values_and_not_finite():
    """A row of equal values is b with eps, NaN without; a NaN or infinity stays in its row; with eps 0 lanes without a
    row add nothing to the weights' gradients."""
    a, g = inputs(5, 40, F32, 2, "wb")
    a["y"][1] = 3.0
    a["y"][2, 7] = float("nan")
    a["y"][3, 1] = float("inf")
    _, h, got = both(a, g, 1e-5, F32)
    assert torch.equal(h[1], a["b"])
    for t in (h, got["dy"]):
        assert torch.isfinite(t[[0, 1, 4]]).all() and not torch.isfinite(t[2]).any() and not torch.isfinite(t[3]).any()
    assert torch.isfinite(got["db"]).all()
    a, g = inputs(3, 24, F32, 4, "wb")
    _, h, got = both(a, g, 0.0, F32)
    check_fwd(a, None, h, 0.0, F32)
    check_bwd(got, a, g, 0.0, F32)
    a["y"][1] = 3.0
    _, h, _ = both(a, g, 0.0, F32)
    assert torch.isnan(h[1]).all() and torch.isfinite(h[[0, 2]]).all()


@pytest.mark.gpu
def test_residual_in_place_and_shapes():
    a, _ = inputs(6, 64, BF16, 6, "xwb")
    d = to_dev(a)
    shape = (2, 3, 64)
    x = d["x"].view(shape).clone()
    want = kda.kda_layer_norm_fwd(d["y"].view(shape), x=d["x"].view(shape), w=d["w"], b=d["b"])
    r, h = kda.kda_layer_norm_fwd(d["y"].view(shape), x=x, w=d["w"], b=d["b"], r=x)
    assert r is x and torch.equal(r, want[0]) and torch.equal(h, want[1]) and h.shape == shape


@pytest.mark.gpu
def test_graph():
    a, g = inputs(300, 264, BF16, 7, "xwb")
    a2, _ = inputs(300, 264, BF16, 8, "xwb")
    d, d2, e = to_dev(a), to_dev(a2), to_dev(g)
    st = {k: v.clone() for k, v in d.items()}

    def call(s):
        r, h = kda.kda_layer_norm_fwd(s["y"], x=s["x"], w=s["w"], b=s["b"])
        o = kda.kda_layer_norm_bwd(s["y"], e["dh"], e["dr"], x=s["x"], w=s["w"])
        return [r, h, o["dy"], o["dw"], o["db"]]

    call(st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(st)
    for s in (d, d2, d, d2):
        for k, v in st.items():
            v.copy_(s[k])
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, call(s)):
            assert torch.equal(p, q)


# ----------------------------------------------------------------------------- refusals (no GPU)
@pytest.fixture(scope="module")
def lib():
    try:
        return kda.load_library()
    except RuntimeError as e:
        pytest.skip(str(e))


NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, ALIAS = 1, 2, 3, 4, 5, 6
AT = {k: (1 << 40) + (i << 30) for i, k in enumerate("y x w b r h dr dh dy dw db ws".split())}


def call(lib, which, **over):
    v = dict(dtype=0, rows=100, D=64, eps=1e-5, bytes=1 << 29)
    v.update(AT)
    v.update(over)
    p = lambda *names: [None if v[n] is None else ctypes.c_void_p(v[n]) for n in names]   # noqa: E731
    head = [v[k] for k in ("dtype", "rows", "D", "eps")]
    if which == "fwd":
        return lib.kda_layer_norm_fwd(*head, *p("y", "x", "w", "b", "r", "h"), None)
    return lib.kda_layer_norm_bwd(*head, *p("y", "x", "w", "dr", "dh", "dy", "dw", "db", "ws"), v["bytes"], None)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), DTYPE), (dict(rows=0), SHAPE), (dict(rows=(1 << 40) + 1), SHAPE), (dict(D=12), SHAPE), (dict(D=8200), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=float("nan")), SHAPE), (dict(y=None), NULL), (dict(x=AT["x"] + 2), ALIGN)])
def test_refusals_of_both(lib, over, status):
    for which in ("fwd", "bwd"):
        assert call(lib, which, **over) == status, which


def test_refusals_of_each(lib):
    assert call(lib, "fwd", h=None) == NULL and call(lib, "fwd", r=None) == NULL and call(lib, "fwd", x=None) == NULL
    assert call(lib, "bwd", dh=None) == NULL and call(lib, "bwd", dy=None) == NULL and call(lib, "bwd", x=None) == NULL
    assert call(lib, "fwd", h=AT["y"]) == ALIAS and call(lib, "fwd", r=AT["x"] + 16) == ALIAS and call(lib, "fwd", r=AT["h"]) == ALIAS
    assert call(lib, "bwd", dy=AT["dh"]) == ALIAS and call(lib, "bwd", dw=AT["db"]) == ALIAS
    assert call(lib, "bwd", ws=None) == WORKSPACE and call(lib, "bwd", bytes=8) == WORKSPACE
    size = ctypes.c_size_t(0)
    assert lib.kda_layer_norm_bwd_workspace_size(100, 64, None) == NULL
    assert lib.kda_layer_norm_bwd_workspace_size(100, 60, ctypes.byref(size)) == SHAPE
    assert lib.kda_layer_norm_bwd_workspace_size(100, 64, ctypes.byref(size)) == 0 and size.value >= 2 * 64 * 4


def test_binding_refuses(lib):
    a, g = inputs(2, 8, F32, 0, "xwb")
    with pytest.raises(ValueError):   # on the CPU
        kda.kda_layer_norm_fwd(a["y"])
    with pytest.raises(ValueError):
        kda.kda_layer_norm_fwd(a["y"], r=a["y"])
    with pytest.raises(ValueError):
        kda.kda_layer_norm_bwd(a["y"], g["dh"], g["dr"])
    with pytest.raises(TypeError):
        kda.kda_layer_norm_fwd(a["y"], w=a["w"].double())
