"""Calls from two host threads at once, whose kernels want different amounts of shared memory."""
import threading

import pytest
import torch

from gated_deltanet_02_gb300 import glinattn_selective_scan_packed

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def in_threads(calls, times):
    """Each of `calls` in a thread and on a stream of its own, `times` times; a call returns what has to stay equal."""
    errors, start = [], threading.Barrier(len(calls))
    wants = [[t.clone() for t in call(torch.cuda.current_stream())] for call in calls]
    torch.cuda.synchronize()

    def work(call, want):
        stream = torch.cuda.Stream(DEV)
        try:
            with torch.cuda.stream(stream):
                start.wait()
                for i in range(times):
                    got = call(stream)
                    if i % 50 == 0 or i == times - 1:
                        stream.synchronize()
                        assert all(torch.equal(a, b) for a, b in zip(got, want))
        except Exception as e:  # noqa: BLE001 - reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(calls, wants)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors


def test_packed_scan_of_single_tokens_beside_drafts():
    """fp32 with 32 states: a CTA's buffers are 54 KB for single tokens and 119 KB for drafts of 24 rows."""
    R, D, N = 40, 512, 32
    g = torch.Generator().manual_seed(1)
    A = -torch.rand((D, N), generator=g).to(DEV)

    def scan(q):
        n = R * q
        x, delta = (torch.randn((n, D), generator=g).to(DEV) for _ in range(2))
        B, C = (torch.randn((n, N), generator=g).to(DEV) for _ in range(2))
        pool = torch.randn((R, D, N), generator=g).to(DEV)
        slots = torch.arange(R, dtype=torch.int32, device=DEV)
        start = torch.arange(0, n + 1, q, dtype=torch.int32, device=DEV)
        y = torch.empty_like(x)

        def call(stream):
            return (glinattn_selective_scan_packed(x, delta, B, C, A, pool, slots, start, max_q_len=q, update_state=False, y=y, stream=stream),)
        return call

    in_threads([scan(1), scan(24)], 4000)
