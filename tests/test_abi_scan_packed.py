"""Packed rows of many sequences in the selective scan, without a GPU: what their workspaces ask for."""
import pytest

from test_abi_scan import lib, need, scan  # noqa: F401

ROW = 256  # pieces of a workspace start at multiples of it


@pytest.mark.parametrize("T,C,S,G", [(32768, 2048, 16, 1), (65536, 2048, 16, 1), (8192, 2048, 64, 1), (8192, 4096, 64, 2), (1000, 48, 32, 3), (5, 32, 16, 1)])
def test_gradients_workspace_grows_with_tokens_and_not_with_sequences_times_tokens(lib, T, C, S, G):
    one = need(lib, "dr_scan_workspace", scan(T=T, C=C, G=G, S=S), 0, 1)
    state = C * S * 4
    for n in (1, 2, 3, 7, 16, 31, 32, 63, 64, 100, 124, 200, 250, 253, 256, 300, 512, 1000, 1024, 2048, 4096):
        packed = need(lib, "dr_scan_workspace", scan(T=T, C=C, G=G, S=S, N=n), 1, 1)
        # Of one row: a checkpoint for every 8 tokens and partial sums for every token. Each sequence, and each segment of one, adds at
        # most a checkpoint, the sums of dA, and where any is cut its state and its gradient's: four states, their steps'
        # sums (no more than half a state together) and table entries. Segments are as many as give each of 1024 SIMDs eight waves.
        slots = n + min(T // 8, 8192 // (G * -(-C // G // 32) * S // 16))
        assert packed <= 1.5 * one + 4.5 * slots * state + 12 * (slots + n + 2) + 9 * ROW, (n, packed, one)
    assert packed >= n * state  # (each sequence's own sum of dA)


def test_largest_packed_sizes_are_answered(lib):
    # 2^20 sequences in a row of 2^26 tokens: the sizes are those of the tokens, not refused as those of their product
    assert need(lib, "dr_scan_workspace", scan(T=1 << 26, C=4096, S=64, N=1 << 20), 1, 1) > 0


@pytest.mark.parametrize("T,C,S", [(32768, 2048, 16), (8192, 1024, 32), (20000, 512, 64)])
@pytest.mark.parametrize("backward", [0, 1])
def test_rows_of_many_sequences_are_cut(lib, T, C, S, backward):
    # the lengths are not known on the host, and one sequence may hold nearly all tokens: whatever the number of the others, it is walked in
    # segments of at most 2048 tokens, each of which has a state in the workspace
    for n in (1, 2, 16, 64, 126, 127, 128, 200, 252, 253, 256, 300, 1000, 4096):
        assert need(lib, "dr_scan_workspace", scan(T=T, C=C, S=S, N=n), 1, backward) >= (n + T // 2048) * C * S * 4, n
