"""Plain 64-bit forms of the operators of a state-space block, for the tests, differentiable by
autograd: the selective scan token by token, the short convolution, the layer norm.  The scan
also gives magnitudes: its sums and those of its gradients over absolute values, by which the tests
turn counts of roundings into bounds."""
import torch


def wide(v, D):
    """[..., G, N] -> [..., D, N]: each channel its group's row."""
    return v.repeat_interleave(D // v.shape[-2], dim=-2)


def step_size(dt, bias, softplus):
    v = dt if bias is None else dt + bias
    return torch.logaddexp(v, torch.zeros_like(v)) if softplus else v


def silu(z):
    return z * torch.sigmoid(z)


def scan64(a, softplus):
    """One sequence from a dict of float64 tensors: x, dt [T,D], A [D,N], b, c [T,G,N], S [D,N], and skip, z, dt_bias or
    None.  Returns y [T,D] and the last state."""
    D, h, ys = a["A"].shape[0], a["S"], []
    for t in range(a["x"].shape[0]):
        d = step_size(a["dt"][t], a["dt_bias"], softplus)
        h = torch.exp(d[:, None] * a["A"]) * h + (d * a["x"][t])[:, None] * wide(a["b"][t], D)
        y = (h * wide(a["c"][t], D)).sum(-1)
        if a["skip"] is not None:
            y = y + a["skip"] * a["x"][t]
        ys.append(y if a["z"] is None else y * silu(a["z"][t]))
    return torch.stack(ys) if ys else a["x"].new_zeros(0, D), h


def scan_magnitudes(a, softplus, dy=None, dS=None):
    """The same sums over absolute values: y, S, and with dy (and dS) the gradients' x, dt, A, b, c, skip, z, dt_bias, S.
    Every gradient of a sum of positive terms is the sum of its own terms' sizes; the step size has two parts, of which
    the decay's is negative throughout, so they are asked for apart."""
    p = {k: None if v is None else v.detach().abs().double() for k, v in a.items()}
    A = a["A"].detach().double()
    d = step_size(a["dt"], a["dt_bias"], softplus).detach().abs()
    leaves = {"x": p["x"], "A": A.clone(), "b": p["b"], "c": p["c"], "S": p["S"], "d1": d.clone(), "d2": d.clone()}
    if p["skip"] is not None:
        leaves["skip"] = p["skip"]
    leaves = {k: v.clone().requires_grad_() for k, v in leaves.items()}
    D, h, pre = A.shape[0], leaves["S"], []
    for t in range(d.shape[0]):
        h = torch.exp(leaves["d2"][t][:, None] * leaves["A"]) * h + (leaves["d1"][t] * leaves["x"][t])[:, None] * wide(leaves["b"][t], D)
        y = (h * wide(leaves["c"][t], D)).sum(-1)
        pre.append(y + leaves["skip"] * leaves["x"][t] if "skip" in leaves else y)
    pre = torch.stack(pre) if pre else d
    gate = None if a["z"] is None else silu(a["z"].detach()).abs()
    y = pre if gate is None else pre * gate
    out = {"y": y.detach(), "S": h.detach()}
    if dy is None:
        return out
    loss = (y * dy.abs()).sum() + (0.0 if dS is None else (h * dS.abs()).sum())
    loss = loss + 0.0 * leaves["S"].sum()   # a sequence without tokens
    g = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()), allow_unused=True)))
    g = {k: torch.zeros_like(leaves[k]) if v is None else v.abs() for k, v in g.items()}
    out.update({"d" + k: g[k] for k in ("x", "A", "b", "c")})
    out["dS0"] = g["S"]
    if "skip" in g:
        out["dskip"] = g["skip"]
    slope = torch.sigmoid(a["dt"] if a["dt_bias"] is None else a["dt"] + a["dt_bias"]).detach() if softplus else 1.0
    out["ddt"] = (g["d1"] + g["d2"]) * slope
    if a["dt_bias"] is not None:
        out["ddt_bias"] = out["ddt"].sum(0)
    if a["z"] is not None:
        z = a["z"].detach()
        sg = torch.sigmoid(z)
        out["dz"] = dy.abs() * pre.detach() * sg * (1 + z.abs() * (1 - sg))
    return out


def conv64(x, w, bias, S, act):
    """One sequence: x [T,D], w [D,W], S [W-1,D] in float64.  Returns y [T,D] and the last W - 1 inputs."""
    W, T = w.shape[1], x.shape[0]
    seq = torch.cat([S, x])
    p = sum(w[:, j] * seq[j:j + T] for j in range(W))
    p = p if bias is None else p + bias
    return silu(p) if act == "silu" else p, seq[T:]


def layer_norm64(a, eps):
    """From a dict of float64 tensors y, x, w, b (None where a part is missing): (r, h)."""
    r = a["y"] if a["x"] is None else a["x"] + a["y"]
    u = r - r.mean(-1, keepdim=True)
    h = u / torch.sqrt(u.pow(2).mean(-1, keepdim=True) + eps)
    h = h if a["w"] is None else h * a["w"]
    return r, h if a["b"] is None else h + a["b"]
