"""The operators together, as a layer of a hybrid model uses them: the norm before the block,
projections, the gated delta rule over packed sequences, the norm and gate of every head, the
projection back, and the residual sum with the next block's norm; trained through, and served as
a prompt and then token by token.

Compared with the same layer in 64 bits, all storage fp32.  A stage's error is known against its
own largest value: 2^-14 for the rule and 2^-13 for its gradients (test_gdr_chunk.py), 2^-15 for norms
and products (up to 256 terms of 2^-24 each are 2^-16, and a value divided by its own norm
has it twice).  What the later stages make of it depends on the rows: o's smallest rows are 70 times smaller
than its largest value, and the heads' norm scales them up.  So the tolerances come from the
64-bit layer itself, before any kernel runs: every stage's result, and every gradient that
goes back through it, is moved by its error with a random sign a value, four times over, and a result may be
off by twice the largest move seen (the errors of a stage are themselves worst cases; the second
half is for signs that four draws do not meet).
"""
import pytest
import torch
import torch.nn.functional as F

import chunked_gated_delta_12_amd as kda
from plain_ops import gdr_tokens, norm64

DEV = "cuda:0"
D, HK, HV, DK, DV, EPS = 128, 2, 4, 32, 64, 1e-6


def weights(seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    w = dict(wq=n(D, HK * DK), wk=n(D, HK * DK), wv=n(D, HV * DV), wz=n(D, HV * DV), wa=n(D, HV), wb=n(D, HV))
    w = {k: t / D ** 0.5 for k, t in w.items()}
    w["wo"] = n(HV * DV, D) / (HV * DV) ** 0.5
    w["n_in"], w["n_out"] = (1 + 0.1 * n(D) for _ in range(2))
    w["n_head"] = 1 + 0.1 * n(DV)
    return w


def gates(w, h):
    """The rule's inputs from the normed rows: unit q and k, log-decay, write strength, and the heads' gate z."""
    rows = h.shape[0]
    unit = lambda t: t / torch.sqrt(t.pow(2).sum(-1, keepdim=True) + EPS)   # noqa: E731
    q, k = (unit((h @ w[n]).view(rows, HK, DK)) for n in ("wq", "wk"))
    v, z = ((h @ w[n]).view(rows, HV, DV) for n in ("wv", "wz"))
    return q, k, v, -F.softplus(h @ w["wa"] - 2), torch.sigmoid(h @ w["wb"]), z


class Rule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, S0, cu):
        ctx.save_for_backward(q, k, v, g, beta, S0, cu)
        return kda.kda_gdr_chunk_fwd(q, k, v, g, beta, S0, cu_seqlens=cu)

    @staticmethod
    def backward(ctx, do, dS_T):
        q, k, v, g, beta, S0, cu = ctx.saved_tensors
        r = kda.kda_gdr_chunk_bwd(q, k, v, g, beta, do.contiguous(), S0, dS_T.contiguous(), cu_seqlens=cu)
        return r["dq"], r["dk"], r["dv"], r["dg"], r["dbeta"], r["dS0"], None


class Norm(torch.autograd.Function):
    """(r, h) of y, x, z, w_post, w_pre; r alone counts where there is no w_pre."""

    @staticmethod
    def forward(ctx, y, x, z, w_post, w_pre, act):
        ctx.save_for_backward(y, x, z, w_post, w_pre)
        ctx.act = act
        return kda.kda_block_norm_fwd(y, x=x, z=z, w_post=w_post, w_pre=w_pre, act=act)

    @staticmethod
    def backward(ctx, dr, dh):
        y, x, z, w_post, w_pre = ctx.saved_tensors
        d = kda.kda_block_norm_bwd(y, dr.contiguous(), None if w_pre is None else dh.contiguous(), x=x, z=z, w_post=w_post,
                                   w_pre=w_pre, act=ctx.act)
        return d["dy"], d["dx"], d["dz"], d["dw_post"], d["dw_pre"], None


def layer(w, x, S0, cu):
    """(residual stream, the next block's input, last states) on the GPU."""
    _, h = Norm.apply(x, None, None, None, w["n_in"], "sigmoid")
    q, k, v, g, beta, z = gates(w, h)
    o, S = Rule.apply(*(t.contiguous()[None] for t in (q, k, v, g, beta)), S0, cu)
    y, _ = Norm.apply(o[0], None, z.contiguous(), w["n_head"], None, "silu")
    r, h = Norm.apply(y.reshape(-1, HV * DV) @ w["wo"], x, None, None, w["n_out"], "sigmoid")
    return r, h, S


def norm_parts(**kw):
    return {**dict(y=None, x=None, z=None, w_post=None, s=None, w_pre=None), **kw}


class Move(torch.autograd.Function):
    """x moved by `fwd` of its largest value, its gradient by `bwd` of its own, signs at random."""

    @staticmethod
    def forward(ctx, x, fwd, bwd, gen):
        ctx.bwd, ctx.gen = bwd, gen
        return Move.by(x, fwd, gen)

    @staticmethod
    def by(x, share, gen):
        sign = torch.randint(0, 2, x.shape, generator=gen, dtype=x.dtype) * 2 - 1
        return x + share * x.detach().abs().max() * sign

    @staticmethod
    def backward(ctx, g):
        return Move.by(g, ctx.bwd, ctx.gen), None, None, None


NORM, RULE, RULE_GRAD = 2.0 ** -15, 2.0 ** -14, 2.0 ** -13


def layer64(w, x, S0, cu, gen=None):
    """The layer in 64 bits; with a generator, every stage moved by its error."""
    def move(t, fwd=NORM, bwd=NORM):
        return t if gen is None else Move.apply(t, fwd, bwd, gen)

    x, S0 = move(x, 0.0), move(S0, 0.0, RULE_GRAD)
    w = {k: move(t, 0.0) for k, t in w.items()}
    _, h = norm64(norm_parts(y=x, w_pre=w["n_in"]), "sigmoid", EPS)
    *rule, z = (move(t) for t in gates(w, move(h)))
    rule = [move(t, 0.0, RULE_GRAD) for t in rule]
    o, S = zip(*(gdr_tokens(*(t[a:b] for t in rule), S0[i], DK ** -0.5) for i, (a, b) in enumerate(zip(cu, cu[1:]))))
    y, _ = norm64(norm_parts(y=move(torch.cat(o), RULE), z=z, w_post=w["n_head"]), "silu", EPS)
    r, h = norm64(norm_parts(y=move(move(y).reshape(-1, HV * DV) @ w["wo"]), x=x, w_pre=w["n_out"]), "sigmoid", EPS)
    return move(r), move(h), move(torch.stack(S), RULE)


def reference(w, x, S0, cu, outs=None):
    """[(result, tolerance)] of r, h, S and, with `outs`, a dict of the same for every gradient."""
    runs = []
    for draw in range(5):
        leaf = {k: t.double().requires_grad_() for k, t in {**w, "x": x, "S0": S0}.items()}
        gen = None if draw == 0 else torch.Generator().manual_seed(100 + draw)
        res = layer64(leaf, leaf["x"], leaf["S0"], cu, gen)
        grads = () if outs is None else torch.autograd.grad(sum((a * b.double()).sum() for a, b in zip(res, outs)), list(leaf.values()))
        runs.append([t.detach() for t in (*res, *grads)])
    both = [(t, 2 * max((m[i] - t).abs().max().item() for m in runs[1:])) for i, t in enumerate(runs[0])]
    return both[:3], dict(zip(leaf, both[3:]))


def near(got, ref, tol, what):
    err = (got.detach().double().cpu() - ref).abs().max().item()
    assert err <= tol, f"{what}: off by {err:.3g}, tolerance {tol:.3g}, largest {ref.abs().max().item():.3g}"


def inputs(lens, seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    cu = [0]
    for t in lens:
        cu.append(cu[-1] + t)
    return n(cu[-1], D), 0.2 * n(len(lens), HV, DK, DV), cu, (n(cu[-1], D), n(cu[-1], D), 0.2 * n(len(lens), HV, DK, DV))


@pytest.mark.gpu
def test_layer_and_its_gradients():
    """A layer over packed sequences, with the gradients of all weights,
    the input and the start states."""
    w, (x, S0, cu, outs) = weights(1), inputs([70, 1, 128, 33], 2)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    leaf = {k: t.to(DEV).requires_grad_() for k, t in {**w, "x": x, "S0": S0}.items()}
    want, grads = reference(w, x, S0, cu, outs)
    got = layer(leaf, leaf["x"], leaf["S0"], c)
    for a, b, what in zip(got, want, ("r", "h", "S")):
        near(a, *b, what)
    dg = torch.autograd.grad(sum((a * b.to(DEV)).sum() for a, b in zip(got, outs)), list(leaf.values()))
    for k, a in zip(leaf, dg):
        near(a, *grads[k], "d" + k)


@pytest.mark.gpu
def test_prompt_then_tokens():
    """A prompt through the chunked rule, then its continuation token by token from the pool of
    states, two requests in a batch with a padded row: the rows of the whole sequence at once."""
    w = {k: t.to(DEV) for k, t in weights(3).items()}
    prompt, more = (65, 30), 5
    full, S0, cu, _ = inputs([p + more for p in prompt], 4)
    ((want, tr), (want_h, th), (want_S, ts)), _ = reference(weights(3), full, S0, cu)
    rows = torch.cat([full[a:a + p] for a, p in zip(cu, prompt)]).to(DEV)
    c = torch.tensor([0, prompt[0], sum(prompt)], dtype=torch.int32, device=DEV)
    r, h, S = layer(w, rows, S0.to(DEV), c)
    pool = torch.full((4, HV, DK, DV), 7.0, device=DEV)
    pool[2], pool[0] = S[0], S[1]
    slots = torch.tensor([2, -1, 0], dtype=torch.int32, device=DEV)
    at = 0
    for i, p in enumerate(prompt):
        near(r[at:at + p], want[cu[i]:cu[i] + p], tr, f"prompt {i}")
        at += p
    for t in range(more):
        x = torch.stack([full[cu[0] + prompt[0] + t], torch.zeros(D), full[cu[1] + prompt[1] + t]]).to(DEV)
        _, hin = kda.kda_block_norm_fwd(x, w_pre=w["n_in"])
        q, k, v, g, beta, z = gates(w, hin)
        o = kda.kda_gdr_step(*(a.contiguous()[:, None] for a in (q, k, v, g, beta)), pool, slots=slots)
        y, _ = kda.kda_block_norm_fwd(o[:, 0], z=z.contiguous(), w_post=w["n_head"], act="silu")
        r, h = kda.kda_block_norm_fwd(y.reshape(3, HV * DV) @ w["wo"], x=x, w_pre=w["n_out"])
        for row, i in ((0, 0), (2, 1)):
            tok = cu[i] + prompt[i] + t
            near(r[row], want[tok], tr, f"token {t} of {i}")
            near(h[row], want_h[tok], th, f"token {t} of {i}")
    near(pool[2], want_S[0], ts, "state 0")
    near(pool[0], want_S[1], ts, "state 1")
    assert (pool[1] == 7).all() and (pool[3] == 7).all()
