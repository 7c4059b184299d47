"""The selective scan's workspace and its pieces, from the size queries (no GPU)."""
import pytest

import chunked_gated_delta_12_amd as kda


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
