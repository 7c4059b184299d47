"""The selective scan's workspace and its pieces, from the size queries (no GPU), and results out of a workspace that
starts as NaN, with more short sequences than the gradients have parts."""
import pytest
import torch

import chunked_gated_delta_12_amd as kda
from test_sel_scan import BF16, DEV, F32, check_bwd, check_fwd, cu_of, inputs, options, spans, to_dev


@pytest.fixture(scope="module", autouse=True)
def lib():
    try:
        return kda.load_library()
    except RuntimeError as e:
        pytest.skip(str(e))


@pytest.mark.parametrize("T", [16384, 16385, 16639, 24577, 65535, 65791, 1 << 20, (1 << 20) + 255, (1 << 30) - 1])
def test_at_most_256_pieces_a_sequence(T):
    """Forwards each piece has D (N + 1) floats."""
    D, N = 64, 16
    pieces, rest = divmod(kda.kda_sel_scan_fwd_workspace_size(1, T, D, N, 1), 4 * D * (N + 1))
    assert rest == 0 and 2 <= pieces <= 256


SIZES = [(4096, 2048, 16, 1), (1 << 20, 256, 64, 2), (100, 64, 8, 1), (65536, 1024, 16, 128), (777, 4096, 32, 1), (3, 1 << 20, 64, 1)]


@pytest.mark.parametrize("T,D,N,G", SIZES)
def test_packed_workspace_is_the_rows_not_the_sequences(T, D, N, G):
    """Forwards a map a piece and a kept state a cut sequence, which is longer than a piece; backwards what the header states, with
    floats a state beside the N."""
    one, mib = kda.kda_sel_scan_fwd_workspace_size(1, T, D, N, G, True), 1 << 20
    B = G * -(-D // G // 64)
    for n in (1, 10, max(1, T // 16), T, 2 * T):
        if n * B >= 1 << 23:
            continue
        assert kda.kda_sel_scan_fwd_workspace_size(n, T, D, N, G, True) <= 2 * one
        size = kda.kda_sel_scan_bwd_workspace_size(n, T, D, N, G, True)
        assert size <= T * (D * (N + 1) / 4 + 8 * N * B) + 24 * D * (N + 2) * max(1, T / 64) + (N + 2) / 2 * mib + 256, n


@pytest.mark.parametrize("nseq,T", [(1, 4096), (4096, 1), (1000, 33), (64, 4096)])
def test_dense_workspace(nseq, T):
    D, N, mib = 1024, 16, 1 << 20
    size = kda.kda_sel_scan_bwd_workspace_size(nseq, T, D, N, 1)
    assert size <= nseq * T * (D * (N + 1) / 4 + 8 * N * 16) + 24 * D * (N + 2) * max(1, nseq * T / 32) + (N + 2) / 2 * mib + 256


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T,D,G", [(1, 1024, 1), (300, 64, 8), (1 << 22, 1024, 1), (70, 1 << 20, 1), (9000, 200, 5)])
def test_sequences_that_are_enough_for_the_header(T, D, G, packed):
    nseq = ((1 << 24) - 1) // (G * -(-D // G // 64)) - 2048
    for size in (kda.kda_sel_scan_fwd_workspace_size, kda.kda_sel_scan_bwd_workspace_size):
        assert nseq < 1 or size(nseq, T, D, 16, G, packed) >= 0


def poisoned(nbytes):
    return torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV)   # as fp32 NaN


def results(x, d, dy, dS, lens, dtype, in_place):
    B, rows, D = x["x"].shape
    N, n = x["A"].shape[1], len(lens) if lens else B
    size = (n, rows, D, N, x["b"].shape[2], lens is not None)
    args, cu = (d["x"], d["dt"], d["A"], d["b"], d["c"]), cu_of(lens) if lens else None
    S = d["S0"].clone()
    y, S_T = kda.kda_sel_scan_fwd(*args, S, S_T=S if in_place else None, cu_seqlens=cu, workspace=poisoned(kda.kda_sel_scan_fwd_workspace_size(*size)),
                                  **options(d, True))
    got = kda.kda_sel_scan_bwd(*args, dy.to(DEV), d["S0"], dS.to(DEV), cu_seqlens=cu, workspace=poisoned(kda.kda_sel_scan_bwd_workspace_size(*size)),
                               **options(d, True))
    torch.cuda.synchronize()
    sp = spans(B, rows, lens)
    check_fwd(x, y.cpu(), S_T.cpu(), sp, True, dtype)
    check_bwd(got, x, dy, dS, sp, True, dtype)


MANY = [3, 0, 1, 0, 7, 2] * 12 + [200] + [1, 5, 0, 2] * 12 + [70, 130, 0, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,D,N,G", [(1, MANY, 2048, 8, 1), (1, MANY, 1032, 16, 3), (90, 5, 2048, 8, 1), (3, 200, 64, 16, 1), (1, [200, 1, 300], 64, 32, 1)])
def test_many_sequences(B, T, D, N, G, dtype):
    """2,048 channels leave 64 parts of the weights' gradients, which 125 packed sequences and 90 of equal length share; sequences
    cut and not cut side by side, the last state over the first."""
    print(f"scan many B={B} T={T if isinstance(T, int) else len(T)} D={D} N={N} G={G} {dtype}", flush=True)
    lens, rows = (T, sum(T)) if isinstance(T, list) else (None, T)
    n = len(lens) if lens else B
    x = inputs(B, rows, D, N, G, dtype, 21, "skip z dt_bias S0", True, n)
    gen = torch.Generator().manual_seed(8)
    dy, dS = torch.randn(B, rows, D, generator=gen).to(dtype), 0.3 * torch.randn(n, D, N, generator=gen)
    results(x, to_dev(x), dy, dS, lens, dtype, True)
