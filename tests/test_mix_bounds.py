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


MANY = 2 ** 32                                               # added to a size: the same in the low 32 bits


def test_sizes_beyond_32_bits_are_refused():
    t = torch.bfloat16
    for call in (lambda k: sq.sq_conv_bytes(t, 256 + k[0], 4 + k[1], 2 + k[2], 40), lambda k: sq.sq_ssm_scan_bytes(t, 256 + k[0], 16 + k[1], 2, 2 + k[2], 40),
                 lambda k: sq.sq_ssm_scan_bytes(t, 256 + k[0], 16, 2 + k[1], 2 + k[2], 40, backward=True),
                 lambda k: sq.sq_delta_scan_bytes(sq.SQ_FORM_GDN, t, 4 + k[0], 4, 128 + k[1], 128, 2 + k[2], 40),
                 lambda k: sq.sq_delta_scan_bytes(sq.SQ_FORM_GDN, t, 4, 4 + k[0], 128, 128 + k[1], 2 + k[2], 40)):
        assert call((0, 0, 0)) >= 0
        for i in range(3):
            for much in (MANY, -MANY, 2 ** 31):
                with pytest.raises(ValueError):
                    call([much if j == i else 0 for j in range(3)])
    assert sq.sq_norm_bytes(100, 256) >= 0
    with pytest.raises(ValueError):
        sq.sq_norm_bytes(100, 256 + MANY)


class Claims:
    """What a call reads of a tensor before it makes its configuration (a real one of these sizes would take gigabytes)."""

    is_cuda, dtype, device = True, torch.bfloat16, torch.device("cuda:0")

    def __init__(self, *shape):
        self.shape = torch.Size(shape)


def test_tensors_beyond_32_bits_are_refused():
    x, w = Claims(2, MANY + 256), Claims(MANY + 256, 4)
    for call in (lambda: sq.sq_conv(x, w, x), lambda: sq.sq_conv_bwd(x, w, x, x), lambda: sq.sq_conv_step(x, w, x, x),
                 lambda: sq.sq_ssm_scan(x, x, Claims(MANY + 256, 16), Claims(2, 1, 16), x, x), lambda: sq.sq_cache_write(x, x, Claims(8, 4)),
                 lambda: sq.sq_cache_read(x, Claims(8, 4), x)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_stream_lookup_without_torchs_short_calls(monkeypatch):
    """The handle of the current stream and the current device come from torch's public calls where the short ones are missing."""
    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(sq, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)
    got = []
    sq._call(lambda *args: got.append(args) or 0, "call", torch.device("cuda:3"), None, 5)
    assert got == [(5, 77)]
