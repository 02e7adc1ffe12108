"""Host-only checks of what room the gated delta rule's segments take: what sequences that are cut can use of it,
not more for each sequence of a batch."""
import ctypes

import pytest

from linear_recurrent_sequence_mamba_amd import binding as m3


def _sizes(B, T, hk, hv, dk, dv, packed):
    lib = m3.library()
    d = m3.m3_delta_dims(B, T, hk, hv, dk, dv, m3.M3_BF16, 0.125, 0, 0, 0, 0, 0)
    return [f(ctypes.byref(d), packed) for f in (lib.m3_delta_scan_workspace_size,
                                                 lib.m3_delta_scan_backward_workspace_size)]


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("packed", [0, 1])
def test_segments_take_room_by_rows(dk, dv, packed):
    """A segment has at least 8 chunks of 64 tokens, so a batch has at most rows / 512 that are not their sequence's
    last.  Of each a state, a map of three 16-bit parts and a decay are kept, in the scan also the state before
    the sequence."""
    for B in (1, 2, 61, 1024, 4096, 100000):
        for T in (1, 511, 512, 513, 4100, 16384, 65536):
            for hv in (1, 16, 32):
                slots = T // 64 + B if packed else B * -(-T // 64)
                if slots * hv >= 1 << 22:
                    continue
                rows = T if packed else B * T
                chunks = (4096 + 320, (dk + 64) * dv)
                for n, c, states in zip(_sizes(B, T, 1, hv, dk, dv, packed), chunks, (2, 1)):
                    most = rows // 512 * hv * (states * 4 * dk * dv + 6 * dk * dk + 4)
                    assert 4 * c * slots * hv <= n <= 4 * c * slots * hv + most, (B, T, hv)


def test_many_short_sequences():
    """4096 sequences of 16 tokens: less than a tenth beside what their chunks take."""
    for n, c in zip(_sizes(4096, 65536, 32, 32, 128, 128, 1), (4096 + 320, 192 * 128)):
        chunks = 4 * c * (65536 // 64 + 4096) * 32
        assert chunks <= n <= 1.4 * chunks
