"""The operators of a state-space block beside the delta rules: the short causal convolution
(forward, backward, token by token), the selective scan (forward, backward, token by token)
and the layer norm with its residual sum (forward, backward).

Short convolution, per channel, with W taps and the W - 1 inputs before the first as state:
    y_t = act(bias + sum_j w_j x_{t-W+1+j}),   act the identity or silu
Selective scan, per channel d with N states, its group's b_t and c_t [N], from a start state h:
    delta_t = softplus(dt_t + dt_bias)  (or dt_t + dt_bias)
    h_n <- exp(delta_t A_n) h_n + delta_t b_t,n x_t;   y_t = (sum_n c_t,n h_n + skip x_t) silu(z_t)
Layer norm, per row:
    r = x + y;   h = (r - mean(r)) / sqrt(mean((r - mean(r))^2) + eps) w + b

Sequences of different lengths come packed, one behind another, with their offsets.
"""
import math

import torch

own = False

EPS = 1e-5
PIECE = 128   # tokens a piece in the plain scan


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # one long document through a layer of 2,048 channels, the state kept for the decode that follows
        dict(name="scan_prefill_64k", op="scan_fwd", dtype="bf16", lens="65536", D=2048, N=16, G=1, s0=False, z=True, skip=True, softplus=True),
        # a serving batch of prompts and of prompts' next pieces: each from its own state, packed
        dict(name="scan_prefill_ragged", op="scan_fwd", dtype="bf16", lens="1,37,512,1000,2049,4096,333,64,8192,100",
             D=2048, N=16, G=1, s0=True, z=True, skip=True, softplus=True),
        # a small layer in 32 bits with two groups, its length no multiple of anything
        dict(name="scan_small_f32", op="scan_fwd", dtype="f32", lens="1000,1000", D=256, N=32, G=2, s0=True, z=False, skip=True, softplus=True),
        # the backward pass of a training step, 4,096 tokens a sequence
        dict(name="scan_train_bwd", op="scan_bwd", dtype="bf16", lens=",".join(["4096"] * 8), D=2048, N=16, G=1, s0=False, z=True, skip=True, softplus=True),
        # the same over documents packed into one row, in 32 bits, the state passed between pieces of a long one
        dict(name="scan_train_bwd_ragged_f32", op="scan_bwd", dtype="f32", lens="2048,1,700,1347", D=512, N=16, G=1, s0=True, z=True, skip=True, softplus=True),
        # one token for each of 256 running requests, their states in a pool
        dict(name="scan_decode_b256", op="scan_step", dtype="bf16", B=256, T=1, D=2048, N=16, G=1, z=True, skip=True, softplus=True),
        # queries, keys and values of 16 heads of 128 channels over one long document
        dict(name="conv_prefill_64k", op="conv_fwd", dtype="bf16", lens="65536", D=6144, W=4, bias=False, act="silu", s0=False),
        # the backward pass over documents packed into one row, the state passed between pieces of a long one
        dict(name="conv_train_bwd_ragged", op="conv_bwd", dtype="bf16", lens="8192,1,2,4700,16384,3489", D=2048, W=4, bias=True, act="silu", s0=True),
        # up to six proposed tokens a request, how many varies
        dict(name="conv_verify_b32", op="conv_step", dtype="bf16", B=32, T=6, D=6144, W=4, bias=True, act="silu"),
        # the rows of a long document between two blocks
        dict(name="layer_norm_64k", op="ln_fwd", dtype="bf16", rows=65536, D=2048, x=True, w=True, b=True),
        # one decode step's rows between two blocks, in 32 bits: latency
        dict(name="layer_norm_small_f32", op="ln_fwd", dtype="f32", rows=7, D=1000, x=True, w=True, b=True),
        # the backward pass between two blocks of a training step
        dict(name="layer_norm_bwd", op="ln_bwd", dtype="bf16", rows=16384, D=2048, x=True, w=True, b=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_lens(rng, most):
    total = _log(rng, 1, most)
    lens, left = [], total
    for _ in range(rng.choice([1, 1, 2, 5, 12])):
        n = min(left, _log(rng, 1, total))   # none left: a request that waits
        lens.append(n)
        left -= n
    return ",".join(map(str, lens))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step", "conv_fwd", "conv_bwd", "conv_step", "ln_fwd", "ln_bwd"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op in ("ln_fwd", "ln_bwd"):
        c["D"] = 8 * _log(rng, 1, 1024)
        c["rows"] = _log(rng, 1, max(1, (1 << 25) // c["D"]))
        for part in ("x", "w", "b"):
            c[part] = rng.random() < 0.7
        return c
    if op in ("conv_fwd", "conv_bwd", "conv_step"):
        c["D"] = 8 * _log(rng, 1, 1024)
        c["W"] = rng.choice([2, 3, 4, 4])
        c["bias"] = rng.random() < 0.5
        c["act"] = rng.choice(["silu", "silu", "none"])
        if op == "conv_step":
            c["T"] = rng.choice([1, 1, 1, 2, 3, 5, 8])
            c["B"] = _log(rng, 1, 512)
            return c
        c["lens"] = _draw_lens(rng, min(65536, (1 << 26) // c["D"]))
        c["s0"] = rng.random() < 0.5
        return c
    c["G"] = rng.choice([1, 1, 1, 2, 4])
    c["D"] = 8 * c["G"] * _log(rng, 1, 512 // c["G"])
    c["N"] = rng.choice([8, 16, 16, 16, 32, 64])
    for part in ("z", "skip"):
        c[part] = rng.random() < 0.7
    c["softplus"] = rng.random() < 0.8
    if op == "scan_step":
        c["T"] = rng.choice([1, 1, 1, 2, 3, 5, 8])
        c["B"] = _log(rng, 1, min(512, max(1, (1 << 23) // (c["D"] * c["N"]))))
        return c
    c["lens"] = _draw_lens(rng, min(16384, (1 << (29 if op == "scan_bwd" else 30)) // (c["D"] * c["N"])))
    c["s0"] = rng.random() < 0.5
    return c


def _lens(case):
    return [int(t) for t in case["lens"].split(",")]


def work(case):
    es, D, op = 2 if case["dtype"] == "bf16" else 4, case["D"], case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        n, par = case["rows"] * D, 4 * D * (case["w"] + case["b"])
        if op == "ln_fwd":   # y, [x] in; [r,] h out
            return {"bytes": es * n * (2 + 2 * case["x"]) + par, "flops": 8 * n}
        return {"bytes": es * n * (3 + 2 * case["x"]) + 4 * D * (2 * case["w"] + case["b"]), "flops": 16 * n}
    if op in ("conv_fwd", "conv_bwd", "conv_step"):
        W = case["W"]
        if op == "conv_step":
            return {"bytes": es * case["B"] * D * (2 * case["T"] + 2 * (W - 1)) + 4 * D * (W + case["bias"]), "flops": 2 * W * case["B"] * case["T"] * D}
        tok, st = sum(_lens(case)), es * len(_lens(case)) * (W - 1) * D
        if op == "conv_fwd":
            return {"bytes": es * tok * D * 2 + st * (1 + case["s0"]) + 4 * D * (W + case["bias"]), "flops": (2 * W + 4) * tok * D}
        return {"bytes": es * tok * D * 3 + 3 * st * case["s0"] + 8 * D * (W + case["bias"]), "flops": (6 * W + 8) * tok * D}
    N, G = case["N"], case["G"]
    par = 4 * D * (N + case["skip"] + case["softplus"])
    if op == "scan_step":
        tok = case["B"] * case["T"]
        return {"bytes": es * tok * (D * (3 + case["z"]) + 2 * G * N) + 8 * case["B"] * D * N + par, "flops": 7 * tok * D * N}
    tok, st = sum(_lens(case)), 4 * len(_lens(case)) * D * N
    if op == "scan_fwd":
        return {"bytes": es * tok * (D * (3 + case["z"]) + 2 * G * N) + st * (1 + case["s0"]) + par, "flops": 7 * tok * D * N}
    # x, dt, b, c, [z] and y's gradient come in, the gradients of the first five go out; the states' with a start state
    return {"bytes": es * tok * (D * (5 + 2 * case["z"]) + 4 * G * N) + 3 * st * case["s0"] + 2 * par, "flops": 20 * tok * D * N}


# ----------------------------------------------------------------------------- the inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, D = case["op"], case["D"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def normal(*shape, mu=0.0, sigma=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(sigma).add_(mu)

    def uniform(lo, hi, *shape):
        return torch.empty(*shape, device="cuda").uniform_(lo, hi, generator=gen)

    st = dict(case=case)
    if op in ("ln_fwd", "ln_bwd"):
        n = case["rows"]
        st["y"] = normal(n, D, mu=0.1, sigma=0.7).to(dt)
        st["x"] = normal(n, D, mu=0.3, sigma=2.0).to(dt) if case["x"] else None
        st["w"] = normal(D, mu=1.0, sigma=0.1) if case["w"] else None
        st["b"] = normal(D, sigma=0.1) if case["b"] else None
        if op == "ln_bwd":
            st["dh"] = normal(n, D).to(dt)
            st["dr"] = normal(n, D).to(dt) if case["x"] else None
        return st

    step = op in ("conv_step", "scan_step")
    if step:
        B, T = case["B"], case["T"]
        lead, nstate = (B, T), B + 3
        st["slots"] = torch.randperm(nstate, generator=gen, device="cuda")[:B].to(torch.int32)
        st["ntok"] = torch.randint(1, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32) if T > 1 else None
        st["y"] = torch.zeros(B, T, D, device="cuda", dtype=dt)
    else:
        lens = _lens(case)
        lead, nstate = (1, sum(lens)), len(lens)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        st["cu"] = torch.tensor(cu, device="cuda", dtype=torch.int32)
        st["maxlen"] = max(lens)
    st["x"] = normal(*lead, D).to(dt)
    if op in ("conv_fwd", "conv_bwd", "conv_step"):
        W = case["W"]
        st["w"] = uniform(-W ** -0.5, W ** -0.5, D, W)
        st["bias"] = normal(D, sigma=0.1) if case["bias"] else None
        st["S"] = normal(nstate, W - 1, D).to(dt) if step or case["s0"] else None
        if op == "conv_bwd":
            st["dy"] = normal(*lead, D).to(dt)
            st["dS_T"] = normal(nstate, W - 1, D).to(dt) if case["s0"] else None
        return st

    N, G = case["N"], case["G"]
    # states that forget fast and states that hardly forget, steps from a thousandth to a tenth
    st["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(normal(D, N, sigma=0.2))
    step_size = torch.exp(uniform(math.log(1e-3), math.log(1e-1), D))
    if case["softplus"]:
        st["dt_bias"] = torch.log(torch.expm1(step_size))
        st["dt"] = normal(*lead, D, sigma=0.5).to(dt)
    else:
        st["dt_bias"] = None
        st["dt"] = (step_size * torch.exp(normal(*lead, D, sigma=0.5))).to(dt)
    st["b"], st["c"] = normal(*lead, G, N).to(dt), normal(*lead, G, N).to(dt)
    st["skip"] = normal(D, mu=1.0, sigma=0.1) if case["skip"] else None
    st["z"] = normal(*lead, D).to(dt) if case["z"] else None
    st["S"] = normal(nstate, D, N, sigma=0.3) if step or case["s0"] else None
    if op == "scan_bwd":
        st["dy"] = normal(*lead, D).to(dt)
        st["dS_T"] = normal(nstate, D, N, sigma=0.3) if case["s0"] else None
    return st


# ----------------------------------------------------------------------------- one pass
def run(st):
    return (_OWN if own else _PLAIN)[st["case"]["op"]](st)


def _act(st):
    return None if st["case"]["act"] == "none" else st["case"]["act"]


def _scan_options(st):
    return dict(skip=st["skip"], z=st["z"], dt_bias=st["dt_bias"], softplus=st["case"]["softplus"])


def _own_scan_fwd(st):
    import chunked_gated_delta_12_amd as kda
    y, S_T = kda.kda_sel_scan_fwd(st["x"], st["dt"], st["A"], st["b"], st["c"], st["S"], cu_seqlens=st["cu"], **_scan_options(st))
    return {"y": y, "S_T": S_T}


def _own_scan_bwd(st):
    import chunked_gated_delta_12_amd as kda
    d = kda.kda_sel_scan_bwd(st["x"], st["dt"], st["A"], st["b"], st["c"], st["dy"], st["S"], st["dS_T"], cu_seqlens=st["cu"],
                             want_dS0=st["S"] is not None, **_scan_options(st))
    return {n: d[n] for n in ("dx", "ddt", "dA", "db", "dc", "dskip", "dz", "ddt_bias", "dS0")}


def _own_scan_step(st):
    import chunked_gated_delta_12_amd as kda
    y = kda.kda_sel_scan_step(st["x"], st["dt"], st["A"], st["b"], st["c"], st["S"], slots=st["slots"], ntok=st["ntok"], y=st["y"],
                              **_scan_options(st))
    return {"y": y, "pool": st["S"]}


def _own_conv_fwd(st):
    import chunked_gated_delta_12_amd as kda
    y, S_T = kda.kda_short_conv_fwd(st["x"], st["w"], st["S"], bias=st["bias"], act=_act(st), cu_seqlens=st["cu"])
    return {"y": y, "S_T": S_T}


def _own_conv_bwd(st):
    import chunked_gated_delta_12_amd as kda
    d = kda.kda_short_conv_bwd(st["x"], st["w"], st["dy"], st["S"], st["dS_T"], bias=st["bias"], act=_act(st), cu_seqlens=st["cu"],
                               want_dS0=st["S"] is not None)
    return {n: d[n] for n in ("dx", "dw", "dbias", "dS0")}


def _own_conv_step(st):
    import chunked_gated_delta_12_amd as kda
    y = kda.kda_short_conv_step(st["x"], st["w"], st["S"], bias=st["bias"], act=_act(st), slots=st["slots"], ntok=st["ntok"], y=st["y"])
    return {"y": y, "pool": st["S"]}


def _own_ln_fwd(st):
    import chunked_gated_delta_12_amd as kda
    r, h = kda.kda_layer_norm_fwd(st["y"], x=st["x"], w=st["w"], b=st["b"], eps=EPS)
    return {"r": r, "h": h}


def _own_ln_bwd(st):
    import chunked_gated_delta_12_amd as kda
    d = kda.kda_layer_norm_bwd(st["y"], st["dh"], st["dr"], x=st["x"], w=st["w"], want_db=st["b"] is not None, eps=EPS)
    return {n: d[n] for n in ("dy", "dw", "db")}


# ----------------------------------------------------------------------------- plain forms: the selective scan
def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _delta(st, dt):
    """The step size of raw dt [..., D] in 32 bits, and its slope."""
    v = dt if st["dt_bias"] is None else dt + st["dt_bias"]
    if not st["case"]["softplus"]:
        return v, torch.ones_like(v)
    return torch.clamp_min(v, 0) + torch.log1p(torch.exp(-v.abs())), _sigmoid(v)


def _pieces(st):
    """The sequences cut into pieces of PIECE tokens: each place's row and whether there is one [pieces, PIECE], each
    piece's sequence, and for the k-th pieces of the sequences their numbers."""
    dev = st["x"].device
    seq, first, kth = [], [], []
    for i, n in enumerate(_lens(st["case"])):
        for k in range(-(-n // PIECE)):
            if k == len(kth):
                kth.append([])
            kth[k].append(len(seq))
            seq.append(i)
            first.append(k * PIECE)
    seq = torch.tensor(seq, device=dev, dtype=torch.long)
    cu = st["cu"].long()
    at = (cu[seq] + torch.tensor(first, device=dev, dtype=torch.long))[:, None] + torch.arange(PIECE, device=dev)
    there = at < cu[seq + 1][:, None]
    return torch.where(there, at, 0), there, seq, [torch.tensor(k, device=dev, dtype=torch.long) for k in kth]


def _spread(x, at, there):
    x = x[0][at].float()
    return torch.where(there.view(*there.shape, *[1] * (x.dim() - 2)), x, torch.zeros((), device=x.device))


def _gather(x, at, there, rows):
    out = torch.zeros(rows + 1, *x.shape[2:], device=x.device)   # places without a row write behind the last
    out[torch.where(there, at, rows)] = x
    return out[None, :rows]


def _wide(v, D):
    """[..., G, N] -> [..., D, N]: each channel its group's row."""
    return v.repeat_interleave(D // v.shape[-2], dim=-2)


def _scan_parts(st):
    at, there, seq, kth = _pieces(st)
    delta, slope = _delta(st, st["dt"][0][at].float())
    zero = torch.zeros((), device=delta.device)
    delta, slope = torch.where(there[..., None], delta, zero), torch.where(there[..., None], slope, zero)   # no row: a step of nothing
    p = dict(at=at, there=there, seq=seq, kth=kth, delta=delta, slope=slope)
    for n in ("x", "b", "c"):
        p[n] = _spread(st[n], at, there)
    return p


def _chain(st, p):
    """Every piece's start state, and the sequences' last states."""
    D, N, A = st["case"]["D"], st["case"]["N"], st["A"]
    P = p["x"].shape[0]
    local = torch.zeros(P, D, N, device=A.device)
    for t in range(PIECE):
        d = p["delta"][:, t, :, None]
        local = torch.exp(d * A) * local + d * p["x"][:, t, :, None] * _wide(p["b"][:, t], D)
    whole = torch.exp(p["delta"].sum(1)[..., None] * A)
    last = torch.zeros(len(_lens(st["case"])), D, N, device=A.device) if st["S"] is None else st["S"].clone()
    start = torch.empty_like(local)
    for k in p["kth"]:
        h = last[p["seq"][k]]
        start[k] = h
        last[p["seq"][k]] = whole[k] * h + local[k]
    return start, last, whole


def _plain_scan_fwd(st):
    D, A, p = st["case"]["D"], st["A"], _scan_parts(st)
    h, last, _ = _chain(st, p)
    y = torch.empty_like(p["x"])
    for t in range(PIECE):
        d = p["delta"][:, t, :, None]
        h = torch.exp(d * A) * h + d * p["x"][:, t, :, None] * _wide(p["b"][:, t], D)
        y[:, t] = (h * _wide(p["c"][:, t], D)).sum(-1)
    if st["skip"] is not None:
        y = y + st["skip"] * p["x"]
    if st["z"] is not None:
        z = _spread(st["z"], p["at"], p["there"])
        y = y * z * _sigmoid(z)
    return {"y": _gather(y, p["at"], p["there"], st["x"].shape[1]).to(st["x"].dtype), "S_T": last}


def _plain_scan_bwd(st):
    case, A, p = st["case"], st["A"], _scan_parts(st)
    D, N, G = case["D"], case["N"], case["G"]
    at, there, x, delta, b, c = p["at"], p["there"], p["x"], p["delta"], p["b"], p["c"]
    h, _, whole = _chain(st, p)
    P, rows, dt = x.shape[0], st["x"].shape[1], st["x"].dtype
    before = []   # the state before each token
    y = torch.empty_like(x)
    for t in range(PIECE):
        before.append(h)
        d = delta[:, t, :, None]
        h = torch.exp(d * A) * h + d * x[:, t, :, None] * _wide(b[:, t], D)
        y[:, t] = (h * _wide(c[:, t], D)).sum(-1)
    dy, dz = _spread(st["dy"], at, there), None
    if st["z"] is not None:
        z = _spread(st["z"], at, there)
        sg = _sigmoid(z)
        whole_y = y if st["skip"] is None else y + st["skip"] * x
        dz = dy * whole_y * sg * (1 + z * (1 - sg))
        dy = dy * z * sg
    # the states' gradients at the pieces' ends: over each piece from nothing, then along the pieces
    lam = torch.zeros(P, D, N, device=A.device)
    for t in range(PIECE - 1, -1, -1):
        lam = torch.exp(delta[:, t, :, None] * A) * (lam + dy[:, t, :, None] * _wide(c[:, t], D))
    mu = torch.zeros(len(_lens(case)), D, N, device=A.device) if st["dS_T"] is None else st["dS_T"].clone()
    end = torch.empty_like(lam)
    for k in p["kth"][::-1]:
        m = mu[p["seq"][k]]
        end[k] = m
        mu[p["seq"][k]] = whole[k] * m + lam[k]
    lam, dA = end, torch.zeros(D, N, device=A.device)
    dx, dd = torch.empty_like(x), torch.empty_like(x)
    db, dc = torch.empty_like(b), torch.empty_like(c)
    for t in range(PIECE - 1, -1, -1):
        d, xt, bt = delta[:, t, :, None], x[:, t, :, None], _wide(b[:, t], D)
        ah = torch.exp(d * A) * before[t]
        dc[:, t] = (dy[:, t, :, None] * (ah + d * xt * bt)).view(P, G, D // G, N).sum(2)
        lam = lam + dy[:, t, :, None] * _wide(c[:, t], D)
        lb = (lam * bt).sum(-1)
        dx[:, t] = delta[:, t] * lb
        db[:, t] = (lam * d * xt).view(P, G, D // G, N).sum(2)
        lah = lam * ah
        dd[:, t] = x[:, t] * lb + (lah * A).sum(-1)
        dA = dA + (d * lah).sum(0)
        lam = torch.exp(d * A) * lam
    ddt = dd * p["slope"]
    out = dict(dA=dA, dskip=None, dz=None, ddt_bias=None, dS0=mu if st["S"] is not None else None)
    if st["skip"] is not None:
        dx = dx + st["skip"] * dy
        out["dskip"] = (dy * x).sum((0, 1))
    if st["dt_bias"] is not None:
        out["ddt_bias"] = ddt.sum((0, 1))
    for n, g in (("dx", dx), ("ddt", ddt), ("db", db), ("dc", dc), ("dz", dz)):
        out[n] = None if g is None else _gather(g, at, there, rows).to(dt)
    return out


def _plain_scan_step(st):
    case, A = st["case"], st["A"]
    D, slots = case["D"], st["slots"].long()
    h, x = st["S"][slots], st["x"].float()
    delta, _ = _delta(st, st["dt"].float())
    for t in range(case["T"]):   # the tokens of one request follow one another
        d = delta[:, t, :, None]
        hn = torch.exp(d * A) * h + d * x[:, t, :, None] * _wide(st["b"][:, t].float(), D)
        y = (hn * _wide(st["c"][:, t].float(), D)).sum(-1)
        if st["skip"] is not None:
            y = y + st["skip"] * x[:, t]
        if st["z"] is not None:
            z = st["z"][:, t].float()
            y = y * z * _sigmoid(z)
        on = torch.ones_like(slots, dtype=torch.bool) if st["ntok"] is None else t < st["ntok"]
        h = torch.where(on[:, None, None], hn, h)
        st["y"][:, t] = torch.where(on[:, None], y.to(st["y"].dtype), st["y"][:, t])
    st["S"][slots] = h
    return {"y": st["y"], "pool": st["S"]}


# ----------------------------------------------------------------------------- plain forms: the short convolution
def _places(st):
    """Each row's sequence, its place there, and the sequence's length."""
    cu = st["cu"].long()
    t = torch.arange(st["x"].shape[1], device=cu.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return t, seq, t - cu[seq], cu[seq + 1] - cu[seq]


def _tap(st, t, seq, place, back):
    """The inputs `back` tokens before each row, from the state where that is before the first."""
    x, W = st["x"][0], st["case"]["W"]
    v = x[torch.clamp_min(t - back, 0)].float()
    if st["S"] is None:
        return torch.where((place >= back)[:, None], v, torch.zeros((), device=x.device))
    return torch.where((place >= back)[:, None], v, st["S"][seq, torch.clamp(W - 1 + place - back, 0, W - 2)].float())


def _last_inputs(st):
    """The last W - 1 inputs of each sequence, its state's among them where it is short."""
    cu, x, W = st["cu"].long(), st["x"][0], st["case"]["W"]
    back = torch.arange(W - 1, device=x.device) - (W - 1)
    at = cu[1:, None] + back
    old = (cu[1:] - cu[:-1])[:, None] + back   # below zero: from the state
    S = torch.zeros(len(cu) - 1, W - 1, x.shape[1], device=x.device, dtype=x.dtype) if st["S"] is None else st["S"]
    from_state = torch.gather(S, 1, torch.clamp(old + W - 1, 0, W - 2)[..., None].expand(-1, -1, x.shape[1]))
    return torch.where((old >= 0)[..., None], x[torch.clamp(at, 0, x.shape[0] - 1)], from_state)


def _pre_activation(st):
    t, seq, place, _ = _places(st)
    W = st["case"]["W"]
    p = torch.zeros(st["x"].shape[1], st["case"]["D"], device=t.device) if st["bias"] is None else st["bias"].expand(len(t), -1)
    for j in range(W):
        p = p + st["w"][:, j] * _tap(st, t, seq, place, W - 1 - j)
    return p


def _plain_conv_fwd(st):
    p = _pre_activation(st)
    if st["case"]["act"] == "silu":
        p = p * _sigmoid(p)
    return {"y": p.to(st["x"].dtype)[None], "S_T": _last_inputs(st)}


def _plain_conv_bwd(st):
    case, W = st["case"], st["case"]["W"]
    t, seq, place, length = _places(st)
    dp = st["dy"][0].float()
    if case["act"] == "silu":
        p = _pre_activation(st)
        sg = _sigmoid(p)
        dp = dp * (sg * (1 + p * (1 - sg)))
    zero, last = torch.zeros((), device=dp.device), len(t) - 1
    dw = torch.stack([(dp * _tap(st, t, seq, place, W - 1 - j)).sum(0) for j in range(W)], 1)
    dx = torch.zeros_like(dp)
    for j in range(W):
        ahead = W - 1 - j
        dx = dx + st["w"][:, j] * torch.where((place + ahead < length)[:, None], dp[torch.clamp_max(t + ahead, last)], zero)
    out = {"dw": dw, "dbias": None if st["bias"] is None else dp.sum(0), "dS0": None}
    if st["S"] is not None:
        i = place - length + W - 1   # the row's place in the last state
        dx = dx + torch.where((i >= 0)[:, None], st["dS_T"][seq, torch.clamp_min(i, 0)].float(), zero)
        cu = st["cu"].long()
        n = (cu[1:] - cu[:-1])[:, None]
        dS0 = []
        for i in range(W - 1):
            g = torch.where(i >= n, st["dS_T"].float()[torch.arange(len(n), device=n.device), torch.clamp_min(i - n[:, 0], 0)], zero)
            for j in range(i + 1):   # state i meets tap j at token i - j
                g = g + st["w"][:, j] * torch.where(i - j < n, dp[torch.clamp(cu[:-1] + i - j, 0, last)], zero)
            dS0.append(g)
        out["dS0"] = torch.stack(dS0, 1).to(st["x"].dtype)
    out["dx"] = dx.to(st["x"].dtype)[None]
    return out


def _plain_conv_step(st):
    case, slots, W = st["case"], st["slots"].long(), st["case"]["W"]
    hist = torch.cat([st["S"][slots], st["x"]], 1)   # the state's inputs, then the tokens'
    n = torch.full_like(slots, case["T"]) if st["ntok"] is None else st["ntok"].long()
    for t in range(case["T"]):
        p = (hist[:, t:t + W].float() * st["w"].t()).sum(1)
        if st["bias"] is not None:
            p = p + st["bias"]
        if case["act"] == "silu":
            p = p * _sigmoid(p)
        st["y"][:, t] = torch.where((t < n)[:, None], p.to(st["y"].dtype), st["y"][:, t])
    at = n[:, None] + torch.arange(W - 1, device=n.device)
    st["S"][slots] = torch.gather(hist, 1, at[..., None].expand(-1, -1, case["D"]))
    return {"y": st["y"], "pool": st["S"]}


# ----------------------------------------------------------------------------- plain forms: the layer norm
def _normed(st):
    r = st["y"].float()
    if st["x"] is not None:
        r = r + st["x"].float()
    u = r - r.mean(-1, keepdim=True)
    rho = torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)
    return r, u * rho, rho


def _plain_ln_fwd(st):
    r, h, _ = _normed(st)
    if st["w"] is not None:
        h = h * st["w"]
    if st["b"] is not None:
        h = h + st["b"]
    return {"r": None if st["x"] is None else r.to(st["y"].dtype), "h": h.to(st["y"].dtype)}


def _plain_ln_bwd(st):
    _, u, rho = _normed(st)
    dh = st["dh"].float()
    t = dh if st["w"] is None else dh * st["w"]
    dy = rho * (t - t.mean(-1, keepdim=True) - u * (t * u).mean(-1, keepdim=True))
    if st["dr"] is not None:
        dy = dy + st["dr"].float()
    return {"dy": dy.to(st["y"].dtype), "dw": None if st["w"] is None else (dh * u).sum(0), "db": None if st["b"] is None else dh.sum(0)}


_OWN = dict(scan_fwd=_own_scan_fwd, scan_bwd=_own_scan_bwd, scan_step=_own_scan_step, conv_fwd=_own_conv_fwd, conv_bwd=_own_conv_bwd,
            conv_step=_own_conv_step, ln_fwd=_own_ln_fwd, ln_bwd=_own_ln_bwd)
_PLAIN = dict(scan_fwd=_plain_scan_fwd, scan_bwd=_plain_scan_bwd, scan_step=_plain_scan_step, conv_fwd=_plain_conv_fwd,
              conv_bwd=_plain_conv_bwd, conv_step=_plain_conv_step, ln_fwd=_plain_ln_fwd, ln_bwd=_plain_ln_bwd)


# ----------------------------------------------------------------------------- from the definitions, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        return _exact_ln(st)
    if op in ("conv_fwd", "conv_bwd"):
        return _exact_conv(st)
    if op == "conv_step":
        return _exact_conv_step(st)
    if op == "scan_step":
        return _exact_scan_step(st)
    return _exact_scan(st)


def _exact_ln(st):
    """Autograd through the definition."""
    bwd = st["case"]["op"] == "ln_bwd"
    a = {n: None if st[n] is None else st[n].double().requires_grad_(bwd) for n in ("y", "x", "w", "b")}
    r = a["y"] if a["x"] is None else a["x"] + a["y"]
    h = (r - r.mean(-1, keepdim=True)) / torch.sqrt(r.var(-1, unbiased=False, keepdim=True) + EPS)
    h = h if a["w"] is None else h * a["w"]
    h = h if a["b"] is None else h + a["b"]
    if not bwd:
        return {"r": None if a["x"] is None else r, "h": h}
    loss = (h * st["dh"].double()).sum()
    if st["dr"] is not None:
        loss = loss + (r * st["dr"].double()).sum()
    have = [n for n in ("y", "w", "b") if a[n] is not None]
    got = dict(zip(have, torch.autograd.grad(loss, [a[n] for n in have])))
    return {"dy": got["y"], "dw": got.get("w"), "db": got.get("b")}


def _conv64(seq, w, bias, act, n):
    """The convolution of one row of inputs [W - 1 + n, D] whose first W - 1 are the state's."""
    p = sum(w[:, j] * seq[j:j + n] for j in range(w.shape[1]))
    p = p if bias is None else p + bias
    return p * torch.sigmoid(p) if act == "silu" else p


def _exact_conv(st):
    """Sequence by sequence, autograd through the definition."""
    case, W, bwd = st["case"], st["case"]["W"], st["case"]["op"] == "conv_bwd"
    w = st["w"].double().requires_grad_(bwd)
    bias = None if st["bias"] is None else st["bias"].double().requires_grad_(bwd)
    xs, ss, ys, ends, lo = [], [], [], [], 0
    for i, n in enumerate(_lens(case)):
        x = st["x"][0, lo:lo + n].double().requires_grad_(bwd)
        s = (torch.zeros(W - 1, case["D"], device=x.device, dtype=x.dtype) if st["S"] is None else st["S"][i].double()).requires_grad_(bwd)
        seq = torch.cat([s, x])
        xs.append(x)
        ss.append(s)
        ys.append(_conv64(seq, w, bias, case["act"], n))
        ends.append(seq[n:])
        lo += n
    if not bwd:
        return {"y": torch.cat(ys)[None], "S_T": torch.stack(ends)}
    loss = (torch.cat(ys) * st["dy"][0].double()).sum()
    if st["dS_T"] is not None:
        loss = loss + (torch.stack(ends) * st["dS_T"].double()).sum()
    leaves = xs + ss + [w] + ([] if bias is None else [bias])
    g = torch.autograd.grad(loss, leaves, allow_unused=True)
    g = [torch.zeros_like(leaf) if v is None else v for leaf, v in zip(leaves, g)]
    n = len(xs)
    return {"dx": torch.cat(g[:n])[None], "dw": g[2 * n], "dbias": None if bias is None else g[-1],
            "dS0": torch.stack(g[n:2 * n]) if st["S"] is not None else None}


def _exact_conv_step(st):
    case = st["case"]
    y, pool, w = st["y"].double(), st["S"].double(), st["w"].double()
    bias = None if st["bias"] is None else st["bias"].double()
    ntok = [case["T"]] * case["B"] if st["ntok"] is None else st["ntok"].tolist()
    for i, (slot, n) in enumerate(zip(st["slots"].tolist(), ntok)):
        seq = torch.cat([pool[slot], st["x"][i, :n].double()])
        y[i, :n] = _conv64(seq, w, bias, case["act"], n)
        pool[slot] = seq[n:]
    return {"y": y, "pool": pool}


def _step64(st, h, x, dt, b, c, A, z):
    """One token of sequences side by side: x, dt, z [S, D], b, c [S, G, N], h [S, D, N] in 64 bits."""
    v = dt if st["dt_bias"] is None else dt + st["dt_bias"].double()
    delta = torch.logaddexp(v, torch.zeros_like(v)) if st["case"]["softplus"] else v
    per = st["case"]["D"] // st["case"]["G"]
    wide = lambda u: u.unsqueeze(2).expand(-1, -1, per, -1).reshape(h.shape)   # noqa: E731
    h = (delta.unsqueeze(-1) * A).exp() * h + (delta * x).unsqueeze(-1) * wide(b)
    y = torch.einsum("sdn,sdn->sd", h, wide(c))
    if st["skip"] is not None:
        y = y + st["skip"].double() * x
    if z is not None:
        y = y * z * torch.sigmoid(z)
    return h, y


def _exact_scan_step(st):
    case, A = st["case"], st["A"].double()
    slots, pool, y = st["slots"].long(), st["S"].double(), st["y"].double()
    ntok = torch.full_like(slots, case["T"]) if st["ntok"] is None else st["ntok"].long()
    for t in range(case["T"]):
        on = torch.nonzero(t < ntok)[:, 0]
        at = lambda n: None if st[n] is None else st[n][on, t].double()   # noqa: E731
        pool[slots[on]], y[on, t] = _step64(st, pool[slots[on]], at("x"), at("dt"), at("b"), at("c"), A, at("z"))
    return {"y": y, "pool": pool}


def _exact_scan(st):
    """Token by token, all sequences side by side; backward by autograd through 32 tokens at a time, from their kept states."""
    case, lens, dev = st["case"], _lens(st["case"]), st["x"].device
    D, N, bwd, L = case["D"], case["N"], case["op"] == "scan_bwd", max(_lens(st["case"]))
    if bwd and L * len(lens) * D * N > 1 << 33:
        return None
    cu = st["cu"].tolist()

    def rows(name):
        if st[name] is None:
            return None
        out = torch.zeros(L, len(lens), *st[name].shape[2:], device=dev, dtype=st[name].dtype)
        for i, n in enumerate(lens):
            out[:n, i] = st[name][0, cu[i]:cu[i] + n]
        return out

    def flat(x):
        return torch.cat([x[:n, i] for i, n in enumerate(lens)])[None]

    X = {n: rows(n) for n in ("x", "dt", "b", "c", "z")}
    on = torch.arange(L, device=dev)[:, None] < torch.tensor(lens, device=dev)   # [L, sequences]
    h = torch.zeros(len(lens), D, N, device=dev, dtype=torch.float64) if st["S"] is None else st["S"].double()
    A = st["A"].double()
    full = [min(lens) > t for t in range(L)]

    def one(par, h, a, t):
        hn, y = _step64(dict(st, **par), h, a["x"], a["dt"], a["b"], a["c"], par.get("A", A), a["z"])
        return (hn if full[t] else torch.where(on[t][:, None, None], hn, h)), y

    at64 = lambda t: {n: None if v is None else v[t].double() for n, v in X.items()}   # noqa: E731
    kept, ys = [], None if bwd else torch.zeros(L, len(lens), D, device=dev, dtype=torch.float64)
    for t in range(L):
        if bwd and t % 32 == 0:
            kept.append(h)
        h, y = one({}, h, at64(t), t)
        if not bwd:
            ys[t] = y
    if not bwd:
        return {"y": flat(ys), "S_T": h}
    dY = rows("dy")
    par = {n: st[n].double().requires_grad_() for n in ("A", "skip", "dt_bias") if st[n] is not None}
    total = {n: torch.zeros_like(v) for n, v in par.items()}
    mu = torch.zeros_like(h) if st["dS_T"] is None else st["dS_T"].double()
    grads = {n: torch.zeros(v.shape, device=dev, dtype=torch.float64) for n, v in X.items() if v is not None}
    for k in range(len(kept) - 1, -1, -1):
        span = range(32 * k, min(L, 32 * k + 32))
        h0 = kept[k].requires_grad_()
        ins = [{n: None if v is None else v.requires_grad_() for n, v in at64(t).items()} for t in span]
        h, loss = h0, 0
        for a, t in zip(ins, span):
            h, y = one(par, h, a, t)
            loss = loss + (y * dY[t].double()).sum()   # dY is zero where there is no row
        loss = loss + (h * mu).sum()
        leaves = [h0] + list(par.values()) + [a[n] for a in ins for n in grads]
        g = torch.autograd.grad(loss, leaves)
        mu = g[0]
        for n, v in zip(par, g[1:]):
            total[n] += v
        rest = iter(g[1 + len(par):])
        for t in span:
            for n in grads:
                grads[n][t] = next(rest)
    out = {"d" + n: flat(grads[n]) if n in grads else None for n in ("x", "dt", "b", "c", "z")}
    out.update({"d" + n: total.get(n) for n in ("A", "skip", "dt_bias")})
    out["dS0"] = mu if st["S"] is not None else None
    return out
