"""What the convolution, the selective scan and the row cache ask of a program's memory and of its numbers, on the CPU."""
import pytest
import torch

import quantized_delta_rule_02_amd as sq


@pytest.mark.parametrize("n_seq", (1, 4, 64, 1024, 4096))
@pytest.mark.parametrize("C,N,G,T", ((4096, 16, 1, 8190), (256, 64, 2, 515), (4096, 16, 1, 0), (200, 8, 4, 12301)))
def test_scan_gradients_workspace_goes_by_tokens_and_sequences(C, N, G, T, n_seq):
    """The states before every 8th token, two states and three sums a channel for each segment of 32 tokens or more and each sequence, and the
    parts of dB and dC; nothing for tokens that a short sequence does not have."""
    state, slots = 4 * C * N, T // 32 + n_seq
    blocks = G * -(-(C // G) // min(64, 1024 // N))           # of channels, at most 64 each
    most = (T // 8 + 1) * (state + 4 * C) + slots * (2 * state + 12 * C) + blocks * T * 8 * N + 8 * 256
    assert 0 < sq.sq_ssm_scan_bytes(torch.bfloat16, C, N, G, n_seq, T, backward=True) <= most
