"""Plain 64-bit forms of the operators beside KDA, for the tests: the gated delta rule
with one decay a head, token by token, and the block norm, both differentiable by
autograd.  Each also gives magnitudes: the same sums over absolute values, by which the
tests turn counts of roundings into bounds."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # relative, of one rounding
U32 = 2.0 ** -24


def rows(x, i, lo, hi):
    return x[i, lo:hi]


def gdr_tokens(q, k, v, g, beta, S, scale):
    """One sequence: q, k [T,Hk,dk], v [T,Hv,dv], g, beta [T,Hv], S [Hv,dk,dv] in float64.
    Returns o [T,Hv,dv] and the last state."""
    rep = v.shape[1] // q.shape[1]
    q, k = (x.repeat_interleave(rep, 1) for x in (q, k))
    o = []
    for t in range(q.shape[0]):
        A = torch.exp(g[t])[:, None, None] * S
        e = v[t] - torch.einsum("hij,hi->hj", A, k[t])
        S = A + torch.einsum("hi,hj->hij", k[t], beta[t][:, None] * e)
        o.append(scale * torch.einsum("hij,hi->hj", S, q[t]))
    return torch.stack(o) if o else v.new_zeros((0,) + v.shape[1:]), S


def gdr_magnitude(q, k, v, g, beta, S, scale):
    """The same recurrence over absolute values with every difference a sum: (o, S) bounds."""
    rep = v.shape[1] // q.shape[1]
    q, k = (x.abs().repeat_interleave(rep, 1) for x in (q, k))
    S, o = S.abs(), []
    for t in range(q.shape[0]):
        A = torch.exp(g[t])[:, None, None] * S
        e = v[t].abs() + torch.einsum("hij,hi->hj", A, k[t])
        S = A + torch.einsum("hi,hj->hij", k[t], beta[t].abs()[:, None] * e)
        o.append(abs(scale) * torch.einsum("hij,hi->hj", S, q[t]))
    return torch.stack(o) if o else v.new_zeros((0,) + v.shape[1:]), S


def gdr_inputs(lead, Hk, Hv, dk, dv, dtype, seed, gmu=-3.0):
    """Seeded inputs [*lead, H, d] on the CPU: unit queries and keys, g <= 0, beta in (0, 1)."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731

    def unit(H):
        x = n(*lead, H, dk) + 0.5 * n(H, dk)
        return (x / x.norm(dim=-1, keepdim=True)).to(dtype)

    x = dict(q=unit(Hk), k=unit(Hk), v=n(*lead, Hv, dv).to(dtype))
    x["g"] = -torch.exp(2 * n(Hv)) * torch.nn.functional.softplus(n(*lead, Hv) + gmu)
    x["beta"] = torch.sigmoid(n(*lead, Hv))
    return x


def norm64(a, act, eps):
    """The block norm from a dict of float64 tensors (None where a part is missing): (r, h)."""
    def rms(x, w):
        return x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * w

    r = a["y"] if a["w_post"] is None else rms(a["y"], a["w_post"])
    if a["z"] is not None:
        r = r * torch.sigmoid(a["z"]) * (a["z"] if act == "silu" else 1.0)
    if a["s"] is not None:
        r = r * a["s"]
    if a["x"] is not None:
        r = r + a["x"]
    return r, None if a["w_pre"] is None else rms(r, a["w_pre"])


def close(got, ref, dtype, mag, roundings, what=""):
    """|got - ref| <= half a step of the storage type at ref + roundings fp32 roundings of mag."""
    got, ref = got.detach().double().cpu(), ref.detach()
    mag = mag if torch.is_tensor(mag) else torch.full_like(ref, mag)
    # a result rounded up to the next binade steps at the larger value: the half step is taken at ref plus the error
    tol = roundings * U32 * mag
    tol = tol + HALF_STEP[dtype] * (ref.abs() + tol) + 1e-37
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = torch.argmax(((got - ref).abs() / tol).nan_to_num(math.inf)).item()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off; worst at {i}: got "
                             f"{got.reshape(-1)[i]:.9g}, want {ref.reshape(-1)[i]:.9g}, tolerance {tol.reshape(-1)[i]:.3g}")
