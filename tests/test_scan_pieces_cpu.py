"""When the packed scan runs long requests in pieces, seen by the workspace that it asks for."""
import ctypes

import pytest

from gated_deltanet_02_gb300 import glinattn as G


def workspace(num_req, num_tok, max_q_len, channels, state=16):
    args = G.ScanPackedArgs(in_dtype=G.BF16, out_dtype=G.BF16, num_req=num_req, num_tok=num_tok, max_q_len=max_q_len, channels=channels,
                            state=state)
    return G.library().glinattn_selective_scan_packed_workspace_size(ctypes.byref(args))


@pytest.mark.parametrize("channels,lengths", [(2048, (1 << 12, 1 << 15)), (256, (1 << 12, 1 << 18, 1 << 20)), (64, (1 << 11, 1 << 20))])
def test_long_requests_of_few_channels_are_run_in_pieces(channels, lengths):
    for n in lengths:
        pieces = n // 512
        assert workspace(1, n, n, channels) >= pieces * channels * (2 * 16 + 1) * 4


@pytest.mark.parametrize("channels,lengths", [(4096, (1 << 13, 1 << 20)), (2048, (1 << 17, 1 << 18, 1 << 20, 1 << 24)), (256, (1 << 23,)), (64, (1 << 24,))])
def test_requests_of_too_many_pieces_are_run_whole(channels, lengths):
    """Each piece reads the ends of all before it: beyond some length that is more than the SMs that idle otherwise."""
    for n in lengths:
        assert workspace(1, n, n, channels) == 0
