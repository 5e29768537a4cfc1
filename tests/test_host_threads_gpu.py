"""Calls from several host threads at once, whose kernels want different amounts of shared memory: the limit that a launch
needs is a property of the kernel, which all threads share."""
import ctypes
import threading

import pytest
import torch

from gated_deltanet_02_gb300 import glinattn as G

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def in_threads(calls, times):
    """The C calls (function, argument struct), each in a thread and on a stream of its own; every one has to succeed."""
    refused, streams = [], []
    start = threading.Barrier(len(calls))

    def work(f, args, stream):
        torch.cuda.set_device(DEV)
        start.wait()
        bad = sum(f(ctypes.byref(args), stream.cuda_stream) != 0 for _ in range(times))
        if bad:
            refused.append(bad)

    threads = []
    for f, args in calls:
        streams.append(torch.cuda.Stream(DEV))
        threads.append(threading.Thread(target=work, args=(f, args, streams[-1])))
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused, refused


def test_packed_scan_of_single_tokens_beside_drafts():
    """fp32 with 32 states: a CTA's buffers are 54 KB for single tokens and 72 KB for drafts of 11 rows."""
    D, N = 32, 32
    A, pool = torch.zeros((D, N), device=DEV), torch.zeros((1, D, N), device=DEV)
    x, B = torch.zeros((11, D), device=DEV), torch.zeros((11, N), device=DEV)
    ints = torch.tensor([0, 1, 0, 11], dtype=torch.int32, device=DEV)
    f, keep, calls = G.library().glinattn_selective_scan_packed, [], []
    for q in (1, 11, 1, 11):
        y = torch.empty_like(x)
        keep.append(y)
        at = ints.data_ptr() + (0 if q == 1 else 8)
        calls.append((f, G.ScanPackedArgs(in_dtype=G.F32, out_dtype=G.F32, num_req=1, num_tok=q, channels=D, state=N, pool_slots=1, max_q_len=q,
                                          x=x.data_ptr(), delta=x.data_ptr(), Bm=B.data_ptr(), Cm=B.data_ptr(), A=A.data_ptr(),
                                          state_pool=pool.data_ptr(), slot_ids=ints.data_ptr(), q_start=at, y=y.data_ptr())))
    in_threads(calls, 20000)


def test_decode_in_both_types():
    """d = 128: a cluster's buffers hold the token's rows in bf16 or in fp32."""
    H, d = 1, 128
    ones, slots = torch.ones(H, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    f, keep, calls = G.library().glinattn_decode, [], []
    for code, act in ((G.BF16, torch.bfloat16), (G.F32, torch.float32)) * 2:
        x, o, pool = torch.zeros((1, H, d), dtype=act, device=DEV), torch.zeros((1, H, d), dtype=act, device=DEV), torch.zeros((1, H, d, d), device=DEV)
        keep += [x, o, pool]
        calls.append((f, G.DecodeArgs(variant=G.GDN, in_dtype=code, out_dtype=code, num_req=1, heads=H, dk=d, dv=d, pool_slots=1, qk_heads=H,
                                      q=x.data_ptr(), k=x.data_ptr(), v=x.data_ptr(), alpha=ones.data_ptr(), beta=ones.data_ptr(),
                                      state_pool=pool.data_ptr(), slot_ids=slots.data_ptr(), o=o.data_ptr())))
    in_threads(calls, 20000)
