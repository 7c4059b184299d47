"""kda_gdr_step against the token-by-token definition in 64 bits.

Tolerance: every value is a chain of products and sums in fp32.  A sum over dk rows is a
chain of dk/8 in a lane and 3 across lanes; with gam = e^g (the exponential and its
argument's rounding: |g| <= 16 here, so 16 more) and the products around it a token adds at
most dk/8 + 32 roundings, so T tokens at most T (dk/8 + 32), of magnitudes taken from the
same recurrence over absolute values; o is rounded once more to its type.
"""
import ctypes

import pytest
import torch

import chunked_gated_delta_12_amd as kda
from plain_ops import close, gdr_inputs, gdr_magnitude, gdr_tokens

DEV = "cuda:0"


def setup(B, T, Hk, Hv, dk, dv, dtype, seed, P=None):
    x = gdr_inputs((B, T), Hk, Hv, dk, dv, dtype, seed)
    x["S"] = 0.3 * torch.randn(P or B, Hv, dk, dv, generator=torch.Generator().manual_seed(seed + 99))
    return x


def reference(x, b, slot, n, scale):
    a = [x[k][b, :n].double() for k in ("q", "k", "v", "g", "beta")] + [x["S"][slot].double(), scale]
    return gdr_tokens(*a), gdr_magnitude(*a)


def run(x, scale, **kw):
    d = {k: v.to(DEV) for k, v in x.items()}
    o = kda.kda_gdr_step(d["q"], d["k"], d["v"], d["g"], d["beta"], d["S"], scale=scale, **kw)
    torch.cuda.synchronize()
    return o.cpu(), d["S"].cpu()


def check_row(x, o, S, b, slot, n, scale, dtype, dk):
    (o64, S64), (mo, mS) = reference(x, b, slot, n, scale)
    per = n * (dk // 8 + 32)
    close(o[b, :n], o64, dtype, mo, per, f"o of row {b}")
    close(S[slot], S64, torch.float32, mS, per, f"state {slot}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,Hk,Hv,dk,dv", [
    (1, 1, 1, 1, 32, 32), (3, 1, 2, 2, 64, 64), (2, 1, 2, 4, 128, 128), (2, 4, 1, 3, 128, 96),
    (1, 7, 2, 2, 32, 256), (2, 3, 1, 4, 64, 224), (1, 33, 1, 2, 128, 160)])
def test_rows_and_tokens(B, T, Hk, Hv, dk, dv, dtype):
    print(f"step B={B} T={T} Hk={Hk} Hv={Hv} dk={dk} dv={dv} {dtype}", flush=True)
    x = setup(B, T, Hk, Hv, dk, dv, dtype, 7)
    scale = dk ** -0.5
    o, S = run(x, None)
    for b in range(B):
        check_row(x, o, S, b, b, T, scale, dtype, dk)


@pytest.mark.gpu
def test_slots_padding_and_duplicates():
    """A pool larger than the batch; rows padded by slot, by length and by a slot that an
    earlier row has; what is padded keeps its o, what no row names keeps its state."""
    B, T, Hk, Hv, dk, dv, P = 9, 3, 2, 4, 64, 64, 12
    x = setup(B, T, Hk, Hv, dk, dv, torch.bfloat16, 3, P)
    slots = [5, -1, 0, 11, 5, 12, 7, 2, 1 << 30]
    ntok = [3, 3, 1, 9, 3, 2, 0, 2, 1]
    real = {0: 3, 2: 1, 3: 3, 7: 2}
    o0 = torch.full((B, T, Hv, dv), 7.0).to(torch.bfloat16)
    o, S = run(x, 0.25, slots=torch.tensor(slots, dtype=torch.int32, device=DEV),
               ntok=torch.tensor(ntok, dtype=torch.int32, device=DEV), o=o0.to(DEV))
    for b, n in real.items():
        check_row(x, o, S, b, slots[b], n, 0.25, torch.bfloat16, dk)
        assert torch.equal(o[b, n:], o0[b, n:])
    for b in set(range(B)) - set(real):
        assert torch.equal(o[b], o0[b]), b
    for s in set(range(P)) - {slots[b] for b in real}:
        assert torch.equal(S[s], x["S"][s]), s


@pytest.mark.gpu
def test_duplicate_far_behind():
    """The scan for an earlier row of the same slot passes more rows than a wavefront has lanes."""
    B, P = 200, 200
    x = setup(B, 1, 1, 1, 32, 32, torch.float32, 4, P)
    slots = torch.randperm(P, generator=torch.Generator().manual_seed(0)).to(torch.int32)
    slots[150] = slots[3]
    slots[199] = slots[70]
    o, S = run(x, 1.0, slots=slots.to(DEV))
    for b in (0, 3, 70, 149, 151, 198):
        check_row(x, o, S, b, int(slots[b]), 1, 1.0, torch.float32, 32)
    assert not o[150].any() and not o[199].any()


@pytest.mark.gpu
def test_same_tokens_at_once_and_one_by_one():
    x = setup(4, 6, 2, 4, 128, 128, torch.float32, 5)
    o, S = run(x, 1.0)
    d = {k: v.to(DEV) for k, v in x.items()}
    for t in range(6):
        ot = kda.kda_gdr_step(*(d[k][:, t:t + 1].contiguous() for k in ("q", "k", "v", "g", "beta")), d["S"], scale=1.0)
        assert torch.equal(ot.cpu()[:, 0], o[:, t]), t
    assert torch.equal(d["S"].cpu(), S)


@pytest.mark.gpu
def test_decays_at_the_ends():
    """g = 0 keeps the state whole, g = -inf and g below fp32's range forget it; beta = 0 and
    k = 0 write nothing; a NaN in one head stays there."""
    x = setup(5, 1, 1, 2, 64, 64, torch.float32, 6)
    for b, g in enumerate((0.0, float("-inf"), -1e4, -104.0, -0.5)):
        x["g"][b] = g
    x["beta"][0] = 0.0
    x["k"][4] = 0.0
    x["v"][4, 0, 1, 5] = float("nan")
    o, S = run(x, 1.0)
    assert torch.equal(S[0], x["S"][0])
    for b in (1, 2):
        e = x["beta"][b, 0][:, None] * x["v"][b, 0]
        want = x["k"][b, 0, 0][None, :, None] * e[:, None, :]
        assert torch.equal(S[b], want)
    assert S[4, 0].isfinite().all() and o[4, 0, 0].isfinite().all() and o[4, 0, 1, 5].isnan()


@pytest.mark.gpu
def test_state_past_32_bits():
    """A pool of more than 2^32 bytes and more than 2^31 elements: the last slots are reached."""
    Hv, dk, dv = 16, 128, 128
    P = (1 << 31) // (Hv * dk * dv) + 3
    S = torch.zeros(P, Hv, dk, dv, device=DEV)
    x = setup(3, 1, 16, Hv, dk, dv, torch.bfloat16, 8)
    slots = [P - 1, 0, P - 3]
    for i, s in enumerate(slots):
        S[s] = x["S"][i].to(DEV)
    d = {k: v.to(DEV) for k, v in x.items()}
    o = kda.kda_gdr_step(d["q"], d["k"], d["v"], d["g"], d["beta"], S, slots=torch.tensor(slots, dtype=torch.int32, device=DEV), scale=1.0)
    o2 = kda.kda_gdr_step(d["q"], d["k"], d["v"], d["g"], d["beta"], d["S"], scale=1.0)
    torch.cuda.synchronize()
    assert torch.equal(o, o2)
    for i, s in enumerate(slots):
        assert torch.equal(S[s], d["S"][i])
    assert not S[1].any() and not S[P - 2].any()


@pytest.mark.gpu
def test_captured_steps():
    """A decode step in a graph, its state and slots changing between replays."""
    x = setup(6, 1, 2, 4, 64, 128, torch.bfloat16, 9, 8)
    d = {k: v.to(DEV) for k, v in x.items()}
    slots = torch.arange(6, dtype=torch.int32, device=DEV)
    o = torch.empty(6, 1, 4, 128, dtype=torch.bfloat16, device=DEV)
    args = [d[k] for k in ("q", "k", "v", "g", "beta")]
    S2, o2 = d["S"].clone(), o.clone()
    kda.kda_gdr_step(*args, S2.clone(), slots=slots)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_gdr_step(*args, d["S"], slots=slots, o=o)
    for i in range(5):
        d["v"].copy_(torch.randn(d["v"].shape, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).to(DEV))
        slots.copy_(((torch.arange(6) + i) % 8).to(torch.int32).to(DEV))
        graph.replay()
        kda.kda_gdr_step(*args, S2, slots=slots, o=o2)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(d["S"], S2), i


# ----------------------------------------------------------------------------- refusals (no GPU)
@pytest.fixture(scope="module")
def lib():
    try:
        return kda.load_library()
    except RuntimeError as e:
        pytest.skip(str(e))


def test_refusals(lib):
    order = ("q", "k", "v", "g", "beta", "S", "slots", "ntok", "o")
    a, base = {}, 1 << 40
    for k in order:
        a[k] = base
        base += 1 << 26

    def call(dtype=0, B=2, T=1, Hk=1, Hv=2, dk=64, dv=64, nslot=4, scale=1.0, **over):
        b = {**a, **over}
        return lib.kda_gdr_step(dtype, B, T, Hk, Hv, dk, dv, nslot, scale,
                                *[None if b[k] is None else ctypes.c_void_p(b[k]) for k in order], None)

    assert call(dtype=2) == 3
    for bad in (dict(B=0), dict(T=0), dict(Hk=0), dict(Hv=0), dict(Hk=2, Hv=3), dict(dk=16), dict(dk=48), dict(dk=256),
                dict(dv=16), dict(dv=48), dict(dv=288), dict(nslot=0), dict(scale=float("inf")), dict(scale=float("nan")),
                dict(B=1 << 30, Hk=1 << 10, Hv=1 << 10)):
        assert call(**bad) == 2, bad
    assert call(slots=None, nslot=1) == 2          # without slots every row needs a state
    for k in ("q", "k", "v", "g", "beta", "S", "o"):
        assert call(**{k: None}) == 1, k
    assert call(q=a["q"] + 2) == 4 and call(slots=a["slots"] + 4) == 4
    assert call(o=a["q"]) == 6 and call(o=a["S"]) == 6 and call(S=a["v"]) == 6 and call(S=a["slots"]) == 6


def test_binding_refusals(lib):
    x = setup(2, 1, 1, 2, 32, 32, torch.float32, 1)
    args = [x[k] for k in ("q", "k", "v", "g", "beta")]
    with pytest.raises(ValueError):
        kda.kda_gdr_step(*args, x["S"])                              # not on the GPU
    with pytest.raises(ValueError):
        kda.kda_gdr_step(*args, x["S"][0])                           # three dimensions
    with pytest.raises(TypeError):
        kda.kda_gdr_step(*args, x["S"], slots=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        kda.kda_gdr_step(*args, x["S"].to(torch.bfloat16))
    with pytest.raises(ValueError):
        kda.kda_gdr_step(x["q"], x["k"], x["v"], x["g"][:1], x["beta"], x["S"])


@pytest.mark.gpu
def test_padded_row_does_not_hold_its_slot():
    """A row without tokens is padding and has no state: the slot that it names belongs to the first
    row behind it that has tokens."""
    B, T, Hk, Hv, dk, dv, P = 7, 2, 1, 2, 64, 96, 6
    x = setup(B, T, Hk, Hv, dk, dv, torch.bfloat16, 12, P)
    slots, ntok = [5, 5, 0, 0, 0, 3, 5], [0, 2, -1, 0, 1, 2, 1]
    real = {1: 2, 4: 1, 5: 2}
    o0 = torch.full((B, T, Hv, dv), 7.0).to(torch.bfloat16)
    o, S = run(x, 0.25, slots=torch.tensor(slots, dtype=torch.int32, device=DEV),
               ntok=torch.tensor(ntok, dtype=torch.int32, device=DEV), o=o0.to(DEV))
    for b, n in real.items():
        check_row(x, o, S, b, slots[b], n, 0.25, torch.bfloat16, dk)
        assert torch.equal(o[b, n:], o0[b, n:])
    for b in set(range(B)) - set(real):
        assert torch.equal(o[b], o0[b]), b
    for s in set(range(P)) - {slots[b] for b in real}:
        assert torch.equal(S[s], x["S"][s]), s
