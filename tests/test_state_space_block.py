"""The operators together, as a state-space block uses them: layer norm, projection, short
convolution, the scan's own projections, the scan with skip and gate, the projection back, and the residual sum
with the next block's norm; trained through, and served as a prompt and then token by token, with
proposed tokens of which some are taken.

Compared with the same block in 64 bits, all storage fp32, by the method of test_gdr_layer.py: every stage's
result, and every gradient that goes back through it, is moved by its error with a random sign a value, four
times over, and a result may be off by twice the largest move seen.  A stage's error against its own largest
value: 2^-15 for norms, products and the convolution (up to 256 terms of 2^-24, twice where a value is divided
by its own norm).  The scan adds at most 11 m + 8 roundings a token to a path whose weight falls by e^-m a token
(m = |delta A|), so what reaches a result is (11 m + 8) min(T, 1 / m) <= 8 T + 11, and 40 for its sums: 1,100
roundings at 130 tokens, 2^-13.9, of magnitudes up to four times the largest value (16 states of either sign):
2^-12, and twice that backwards, where a path is two scans long.
"""
import pytest
import torch

import chunked_gated_delta_12_amd as kda
from plain_state_space import conv64, layer_norm64, scan64
from test_gdr_layer import Move, near

DEV = "cuda:0"
DM, D, N, G, R, W, EPS = 64, 128, 16, 2, 8, 4, 1e-5   # block width, channels, states, groups, rank of the step sizes, taps
OTHER, SCAN, SCAN_GRAD = 2.0 ** -15, 2.0 ** -12, 2.0 ** -11


def weights(seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    w = dict(w_in=n(DM, 2 * D) / DM ** 0.5, w_par=n(D, R + 2 * G * N) / D ** 0.5, w_dt=n(R, D) / R ** 0.5, w_out=n(D, DM) / D ** 0.5)
    w["conv"], w["conv_b"] = (2 * torch.rand(D, W, generator=gen) - 1) * W ** -0.5, 0.1 * n(D)
    w["A"] = -torch.arange(1, N + 1).float() * torch.exp(0.2 * n(D, N))
    w["dt_b"], w["skip"] = n(D) - 4, 1 + 0.1 * n(D)
    for k in ("in", "next"):
        w["n_" + k], w["b_" + k] = 1 + 0.1 * n(DM), 0.1 * n(DM)
    return w


def split(p, w):
    """Step sizes before their softplus, b and c from the scan's projections."""
    dt, b, c = p.split([R, G * N, G * N], -1)
    return dt @ w["w_dt"], b.unflatten(-1, (G, N)), c.unflatten(-1, (G, N))


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, x, w, b):
        ctx.save_for_backward(y, x, w)
        r, h = kda.kda_layer_norm_fwd(y, x=x, w=w, b=b, eps=EPS)
        return (y.clone() if r is None else r), h

    @staticmethod
    def backward(ctx, dr, dh):
        y, x, w = ctx.saved_tensors
        d = kda.kda_layer_norm_bwd(y, dh.contiguous(), None if x is None else dr.contiguous(), x=x, w=w, eps=EPS)
        return d["dy"], None if x is None else d["dy"], d["dw"], d["db"]


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, S0, cu):
        ctx.save_for_backward(x, w, b, S0, cu)
        return kda.kda_short_conv_fwd(x, w, S0, bias=b, act="silu", cu_seqlens=cu)

    @staticmethod
    def backward(ctx, dy, dS):
        x, w, b, S0, cu = ctx.saved_tensors
        d = kda.kda_short_conv_bwd(x, w, dy.contiguous(), S0, dS.contiguous(), bias=b, act="silu", cu_seqlens=cu)
        return d["dx"], d["dw"], d["dbias"], d["dS0"], None


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, b, c, skip, z, dt_b, S0, cu):
        ctx.save_for_backward(x, dt, A, b, c, skip, z, dt_b, S0, cu)
        return kda.kda_sel_scan_fwd(x, dt, A, b, c, S0, skip=skip, z=z, dt_bias=dt_b, cu_seqlens=cu)

    @staticmethod
    def backward(ctx, dy, dS):
        x, dt, A, b, c, skip, z, dt_b, S0, cu = ctx.saved_tensors
        d = kda.kda_sel_scan_bwd(x, dt, A, b, c, dy.contiguous(), S0, dS.contiguous(), skip=skip, z=z, dt_bias=dt_b, cu_seqlens=cu)
        return tuple(d[k] for k in ("dx", "ddt", "dA", "db", "dc", "dskip", "dz", "ddt_bias", "dS0")) + (None,)


def block(w, x, C0, S0, cu):
    """(residual stream, the next block's input, the convolution's and the scan's last states) on the GPU."""
    _, h = Norm.apply(x, None, w["n_in"], w["b_in"])
    u, z = (t.contiguous()[None] for t in (h @ w["w_in"]).chunk(2, -1))
    v, C = Conv.apply(u, w["conv"], w["conv_b"], C0, cu)
    dt, b, c = (t.contiguous() for t in split(v @ w["w_par"], w))
    y, S = Scan.apply(v, dt, w["A"], b, c, w["skip"], z, w["dt_b"], S0, cu)
    r, h = Norm.apply(y[0] @ w["w_out"], x, w["n_next"], w["b_next"])
    return r, h, C, S


def block64(w, x, C0, S0, cu, gen=None):
    def move(t, fwd=OTHER, bwd=OTHER):
        return t if gen is None else Move.apply(t, fwd, bwd, gen)

    x, C0, S0 = move(x, 0.0), move(C0, 0.0), move(S0, 0.0, SCAN_GRAD)
    w = {k: move(t, 0.0, SCAN_GRAD if k in ("A", "skip", "dt_b") else OTHER) for k, t in w.items()}
    _, h = layer_norm64(dict(y=x, x=None, w=w["n_in"], b=w["b_in"]), EPS)
    u, z = (move(t) for t in (move(h) @ w["w_in"]).chunk(2, -1))
    ends = list(zip(cu, cu[1:]))
    v, C = zip(*(conv64(u[a:b], w["conv"], w["conv_b"], C0[i], "silu") for i, (a, b) in enumerate(ends)))
    v = move(torch.cat(v))
    args = [move(t, 0.0, SCAN_GRAD) for t in (v, *(move(t) for t in split(v @ w["w_par"], w)), z)]
    y, S = [], []
    for i, (a, b) in enumerate(ends):
        p = dict(zip(("x", "dt", "b", "c", "z"), (t[a:b] for t in args)), A=w["A"], skip=w["skip"], dt_bias=w["dt_b"], S=S0[i])
        yi, Si = scan64(p, True)
        y.append(yi)
        S.append(Si)
    r, h = layer_norm64(dict(y=move(move(torch.cat(y), SCAN) @ w["w_out"]), x=x, w=w["n_next"], b=w["b_next"]), EPS)
    return move(r), move(h), move(torch.stack(C)), move(torch.stack(S), SCAN)


def reference(w, x, C0, S0, cu, outs=None):
    """[(result, tolerance)] of r, h, C, S and, with `outs`, a dict of the same for every gradient."""
    runs = []
    for draw in range(5):
        leaf = {k: t.double().requires_grad_() for k, t in {**w, "x": x, "C0": C0, "S0": S0}.items()}
        gen = None if draw == 0 else torch.Generator().manual_seed(100 + draw)
        res = block64({k: leaf[k] for k in w}, leaf["x"], leaf["C0"], leaf["S0"], cu, gen)
        grads = () if outs is None else torch.autograd.grad(sum((a * b.double()).sum() for a, b in zip(res, outs)), list(leaf.values()))
        runs.append([t.detach() for t in (*res, *grads)])
    both = [(t, 2 * max((m[i] - t).abs().max().item() for m in runs[1:])) for i, t in enumerate(runs[0])]
    return both[:4], dict(zip(leaf, both[4:]))


def inputs(lens, seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    cu, k = [0], len(lens)
    for t in lens:
        cu.append(cu[-1] + t)
    outs = (n(cu[-1], DM), n(cu[-1], DM), n(k, W - 1, D), 0.2 * n(k, D, N))
    return n(cu[-1], DM), 0.3 * n(k, W - 1, D), 0.2 * n(k, D, N), cu, outs


@pytest.mark.gpu
def test_block_and_its_gradients():
    """A block over packed sequences, with the gradients of all weights, the input and both start states."""
    w, (x, C0, S0, cu, outs) = weights(1), inputs([70, 1, 130, 33], 2)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    leaf = {k: t.to(DEV).requires_grad_() for k, t in {**w, "x": x, "C0": C0, "S0": S0}.items()}
    want, grads = reference(w, x, C0, S0, cu, outs)
    got = block(leaf, leaf["x"], leaf["C0"], leaf["S0"], c)
    for a, b, what in zip(got, want, ("r", "h", "C", "S")):
        near(a, *b, what)
    dg = torch.autograd.grad(sum((a * b.to(DEV)).sum() for a, b in zip(got, outs)), list(leaf.values()))
    for k, a in zip(leaf, dg):
        near(a, *grads[k], "d" + k)


@pytest.mark.gpu
def test_prompt_then_tokens_and_proposals():
    """A prompt, then its continuation from pools of states: tokens one by one with a padded row in the batch, then
    four proposed tokens a request, evaluated on copies of the states; of those three and one are taken."""
    w = {k: t.to(DEV) for k, t in weights(3).items()}
    prompt, one_by_one, proposed, taken = (65, 30), 3, 4, (3, 1)
    full, C0, S0, cu, _ = inputs([p + one_by_one + proposed for p in prompt], 4)
    ((want, tr), (want_h, th), _, _), _ = reference(weights(3), full, C0, S0, cu)
    rows = torch.cat([full[a:a + p] for a, p in zip(cu, prompt)]).to(DEV)
    c = torch.tensor([0, prompt[0], sum(prompt)], dtype=torch.int32, device=DEV)
    r, h, C, S = block(w, rows, C0.to(DEV), S0.to(DEV), c)
    pools = torch.full((4, W - 1, D), 7.0, device=DEV), torch.full((4, D, N), 7.0, device=DEV)
    for pool, state in zip(pools, (C, S)):
        pool[2], pool[0] = state[0], state[1]
    slots = torch.tensor([2, -1, 0], dtype=torch.int32, device=DEV)
    for i, p in enumerate(prompt):
        near(r[sum(prompt[:i]):sum(prompt[:i]) + p], want[cu[i]:cu[i] + p], tr, f"prompt {i}")

    def tokens(t, n, pools, ntok=None):
        """Rows t .. t + n of both requests, [3, n, ..] with a padded row between."""
        x = torch.stack([full[cu[0] + prompt[0] + t:][:n], torch.zeros(n, DM), full[cu[1] + prompt[1] + t:][:n]]).to(DEV)
        ntok = None if ntok is None else torch.tensor([ntok[0], 0, ntok[1]], dtype=torch.int32, device=DEV)
        _, h = kda.kda_layer_norm_fwd(x, w=w["n_in"], b=w["b_in"], eps=EPS)
        u, z = (a.contiguous() for a in (h @ w["w_in"]).chunk(2, -1))
        v = kda.kda_short_conv_step(u, w["conv"], pools[0], bias=w["conv_b"], act="silu", slots=slots, ntok=ntok)
        dt, b, c = (a.contiguous() for a in split(v @ w["w_par"], w))
        y = kda.kda_sel_scan_step(v, dt, w["A"], b, c, pools[1], skip=w["skip"], z=z, dt_bias=w["dt_b"], slots=slots, ntok=ntok)
        return kda.kda_layer_norm_fwd(y @ w["w_out"], x=x, w=w["n_next"], b=w["b_next"], eps=EPS)

    def check(got, t, n):
        for row, i in ((0, 0), (2, 1)):
            at = cu[i] + prompt[i] + t
            near(got[0][row, :n[i]], want[at:at + n[i]], tr, f"tokens from {t} of {i}")
            near(got[1][row, :n[i]], want_h[at:at + n[i]], th, f"tokens from {t} of {i}")

    for t in range(one_by_one):
        check(tokens(t, 1, pools), t, (1, 1))
    kept = [p.clone() for p in pools]
    check(tokens(one_by_one, proposed, [p.clone() for p in pools]), one_by_one, (proposed, proposed))
    assert all(torch.equal(a, b) for a, b in zip(pools, kept))
    check(tokens(one_by_one, proposed, pools, taken), one_by_one, taken)
    # from what was taken on, request 1's next tokens one by one
    for t in range(taken[1], proposed):
        x = tokens(one_by_one + t, 1, pools, (0, 1))
        near(x[0][2], want[cu[1] + prompt[1] + one_by_one + t][None], tr, f"token {t} behind the taken one")
    for pool in pools:
        assert (pool[1] == 7).all() and (pool[3] == 7).all()
