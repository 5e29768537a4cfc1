"""Calls from a host thread that has made no CUDA call before: the library needs no context that someone else made current."""
import threading

import pytest
import torch

import gated_deltanet_02_gb300 as G
from gated_deltanet_02_gb300 import inputs
from paged_helpers import cache_args, dev, paged_case

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


def gpu(c):
    return {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in c.items()}


def prefill(make, variant, **kw):
    c = gpu(make(1, 2, 256, 128, **kw))
    o, s = torch.empty_like(c["v"]), torch.empty((1, 2, 128, 128), device=DEV)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    return lambda: G.glinattn_prefill(c["q"], c["k"], c["v"], c["alpha"], c["beta"], variant=variant, o=o, S_T=s, workspace=ws)[:2]


def decode(d):
    c = gpu(inputs.gdn_decode(4, 2, d, 6, conv=False))
    o = torch.empty_like(c["v"])

    def call():
        c["state_pool"] = c["pool"] * 0 + 1
        G.glinattn_decode(c["q"], c["k"], c["v"], c["alpha"], c["beta"], c["state_pool"], c["slot_ids"], o=o)
        return o, c["state_pool"]
    return call


def attention(d, cache, q_len):
    c = paged_case([(q_len, 100), (1, 40)], 2, d, 16, cache, seed=d)
    g = dev(c)
    args, kw = cache_args(g)
    q = torch.randn((c["num_tok"], 4, d), generator=torch.Generator().manual_seed(1)).to(BF16).to(DEV)
    o, ws = torch.empty_like(q), torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    return lambda: (G.glinattn_paged_attention(q, *args, max_q_len=q_len, o=o, workspace=ws, **kw),)


CALLS = {
    "gla prefill": lambda: prefill(inputs.gla_prefill, G.GLA), "gdn prefill": lambda: prefill(inputs.gdn_prefill, G.GDN, conv=False),
    "decode 128": lambda: decode(128), "decode 64": lambda: decode(64),
    "prompts bf16": lambda: attention(128, "bf16", 60), "prompts e4m3": lambda: attention(64, "e4m3", 60),
    "tokens bf16": lambda: attention(64, "bf16", 1), "tokens e4m3": lambda: attention(128, "e4m3", 1),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_first_call_of_a_thread(name):
    call = CALLS[name]()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    got = []

    def work():
        try:
            got.extend(call())
        except Exception as e:  # noqa: BLE001 - looked at by the test's own thread
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert len(got) == len(want) and all(isinstance(g, torch.Tensor) and torch.equal(g, w) for g, w in zip(got, want)), got
