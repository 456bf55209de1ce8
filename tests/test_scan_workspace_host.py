"""The scan's workspaces (CPU) follow its tensors: batches of many short sequences
keep no partial sum for each of them, whatever the number of states."""
import pytest

import convolution_implicit_gemm_conv2d_amd as cm


# sequences, rows of each, channels, states
MANY = [(131072, 4, 4096, 16), (2048, 64, 4096, 64), (1 << 20, 1, 512, 8), (1 << 24, 1, 16, 16), (4096, 33, 1000, 24), (100_000, 7, 2048, 1), (1 << 20, 0, 4096, 64)]


@pytest.mark.parametrize("S,L,C,N", MANY)
def test_many_short_sequences(S, L, C, N):
    got = cm.conv_scan_bwd_workspace_size(S * L, S, C, N, 1, False, True)
    # a GiB of partial sums of dB and dC, and those of dA of 2^14 workgroups with
    # at most 64 channels each
    assert got <= (1 << 30) + ((1 << 14) + C) * 64 * (N + 2) * 4 + (1 << 20), got
    assert cm.conv_scan_fwd_workspace_size(S * L, S, C, N, 1, False) == 0 or S * L < 2048
    # without kept states those are there, too
    saved = cm.conv_scan_saved_size(S * L, C, N)
    assert 0 <= cm.conv_scan_bwd_workspace_size(S * L, S, C, N, 1, False, False) - got - saved < 16


def test_few_sequences_are_as_before():
    """One launch, a partial sum of dA for each sequence."""
    S, L, C, N = 8, 2048, 2048, 16
    assert cm.conv_scan_bwd_workspace_size(S * L, S, C, N, 1, False, True) == C // 32 * S * L * 2 * N * 4 + S * C * (N + 2) * 4
