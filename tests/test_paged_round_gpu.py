"""A whole speculative round of a hybrid stack, the calls together: drafts through
a Gated DeltaNet layer (verify only) and a softmax layer (cache write, attention
over the paged cache), acceptance, replay of the accepted drafts -- and the next
round over what the first one left."""
import math

import numpy as np
import pytest
import torch

import oracle
from gated_deltanet_02_gb300 import (GDN, glinattn_accept_drafts, glinattn_kv_append, glinattn_kv_gather,
                                     glinattn_paged_attention, glinattn_replay, glinattn_spec_decode, inputs)
from oracle import paged as P

from helpers import TOL_S_BF16, f64, relerr
from paged_helpers import attention_tolerance, cache_args, dev, paged_case, rows_of

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("graph", [False, True])
def test_two_speculative_rounds(cache, graph):
    R, D, V, H, Hkv, d = 6, 3, 500, 8, 2, 128
    hist = [0, 5, 40, 127, 200, 333]
    # room in the page tables for two rounds of D + 1 tokens
    c = paged_case([(0, h + 2 * (D + 1)) for h in hist], Hkv, d, 16, cache, seed=1)
    c["lengths"] = [(D + 1, h + D + 1) for h in hist]
    gen = torch.Generator().manual_seed(2)

    base = inputs.gdn_decode(R, 2, d, 12, seed=3)           # the linear layer's pool: 2 heads
    slots = base["slot_ids"]
    rounds = []
    for k in range(2):
        dr = inputs.spec_drafts(R, D, 2, d, seed=10 + k)
        z = torch.randn((R, D + 1, V), generator=gen) * 2
        target = torch.softmax(z + 0.4 * torch.randn((R, D + 1, V), generator=gen), -1)
        draft = torch.softmax(z[:, :D], -1)
        rounds.append(dict(
            dr=dr, target=target, draft=draft,
            tokens=torch.multinomial(draft.reshape(-1, V), 1, generator=gen).reshape(R, D).to(torch.int32),
            u=torch.rand((R, D + 1), generator=gen),
            k=torch.randn((R * (D + 1), Hkv, d), generator=gen).to(torch.bfloat16),
            v=torch.randn((R * (D + 1), Hkv, d), generator=gen).to(torch.bfloat16),
            q=torch.randn((R * (D + 1), H, d), generator=gen).to(torch.bfloat16)))

    # device buffers of one round, as a captured step would keep them
    g = dev(c)
    args, scales = cache_args(g)
    g["kv_len"].copy_(torch.tensor([h + D + 1 for h in hist], dtype=torch.int32))
    g["q_start"].copy_(torch.arange(R + 1, dtype=torch.int32) * (D + 1))
    to = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    buf = {k: to(v).clone() for k, v in rounds[0].items() if k != "dr"}
    lin = {k: to(v).clone() for k, v in rounds[0]["dr"].items() if v is not None}
    pool, cpool, w = to(base["pool"]).clone(), to(base["conv_pool"]).clone(), to(base["conv_w"])
    sl = to(slots)
    accept = torch.empty(R, dtype=torch.int32, device=DEV)
    drawn = torch.empty((R, D + 1), dtype=torch.int32, device=DEV)
    out = torch.empty((R * (D + 1), H, d), dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def step():
        o_lin = glinattn_spec_decode(lin["q"], lin["k"], lin["v"], lin["alpha"], lin["beta"], pool, sl, None, variant=GDN,
                                     conv_w=w, conv_pool=cpool, qk_l2norm=True, out_dtype=torch.float32, dev_status=status)
        glinattn_kv_append(buf["k"], buf["v"], *args, **scales, dev_status=status)
        glinattn_paged_attention(buf["q"], *args, **scales, max_q_len=D + 1, o=out, dev_status=status)
        glinattn_accept_drafts(buf["target"], buf["draft"], buf["tokens"], buf["u"], accept=accept, tokens=drawn, dev_status=status)
        glinattn_replay(lin["k"], lin["v"], lin["alpha"], lin["beta"], pool, sl, accept, q=lin["q"], variant=GDN, conv_w=w,
                        conv_pool=cpool, qk_l2norm=True, dev_status=status)
        # the accepted drafts and the drawn token's place stay in the cache
        g["kv_len"].sub_(D + 1).add_(accept).add_(1)
        return o_lin

    if graph:
        saved = [t.clone() for t in (pool, cpool, g["kv_len"], g["k_cache"].view(torch.uint8), g["v_cache"].view(torch.uint8))]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured, stream=side):
            step()
        for t, x in zip((pool, cpool, g["kv_len"], g["k_cache"].view(torch.uint8), g["v_cache"].view(torch.uint8)), saved):
            t.copy_(x)

    lengths = list(hist)
    state, conv = f64(base["pool"]), f64(base["conv_pool"])
    for k in range(2):
        rd = rounds[k]
        if k:
            g["kv_len"].add_(D + 1)
            for name in buf:
                buf[name].copy_(rd[name])
            for name in lin:
                lin[name].copy_(rd["dr"][name])
        captured.replay() if graph else step()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        # acceptance
        a, t = P.accept_drafts(rd["target"].numpy(), rd["draft"].numpy(), rd["tokens"].numpy(), rd["u"].numpy())
        assert np.array_equal(accept.cpu().numpy(), a) and np.array_equal(drawn.cpu().numpy(), t)
        # attention over the cache as it is now
        now = {n: (x.cpu() if isinstance(x, torch.Tensor) else x) for n, x in g.items()}
        now["lengths"] = [(D + 1, h + D + 1) for h in lengths]
        now["kv_len"] = torch.tensor([h + D + 1 for h in lengths], dtype=torch.int32)
        qd = rd["q"].double().numpy()
        kr, vr = rows_of(now, "k"), rows_of(now, "v")
        want, mag = P.attention(qd, kr, vr, now["q_start"], now["kv_len"], 1 / math.sqrt(d))
        assert (np.abs(out.double().cpu().numpy() - want) <= attention_tolerance(now, qd, want, mag, 1 / math.sqrt(d))).all()
        # the linear layer: the state after the accepted drafts
        n_slot = state.shape[0]
        wide = np.concatenate([state, np.zeros((R * D,) + state.shape[1:])])
        wide_c = np.concatenate([conv, np.zeros((R * D,) + conv.shape[1:])])
        dst = (n_slot + np.arange(R * D)).reshape(R, D)
        f = {n: f64(x) for n, x in rd["dr"].items()}
        _, wp, wc = oracle.spec_decode(GDN, f["q"], f["k"], f["v"], f["alpha"], f["beta"], wide, slots.tolist(), dst.tolist(),
                                       f64(base["conv_w"]), wide_c, True)
        for r in range(R):
            if a[r]:
                state[int(slots[r])], conv[int(slots[r])] = wp[dst[r, a[r] - 1]], wc[dst[r, a[r] - 1]]
        assert relerr(pool, state) <= TOL_S_BF16
        assert np.array_equal(f64(cpool), conv)
        lengths = [h + int(x) + 1 for h, x in zip(lengths, a)]
        assert g["kv_len"].cpu().tolist() == lengths
    # what is left in the cache of the second round: its accepted rows, read back
    qs = torch.tensor(np.concatenate([[0], np.cumsum([int(x) + 1 for x in a])]), dtype=torch.int32, device=DEV)
    k2, v2 = glinattn_kv_gather(*args[:4], qs, num_tok=int(qs[-1]), **scales)
    at = 0
    for r in range(R):
        n = int(a[r]) + 1
        for got, src in ((k2, rounds[1]["k"]), (v2, rounds[1]["v"])):
            x = src[r * (D + 1):r * (D + 1) + n].double().numpy()
            if cache == "e4m3":
                val, e = P.quantise(x)
                x = val * 2.0 ** e[..., None].astype(np.float64)
            assert np.array_equal(got[at:at + n].double().cpu().numpy(), x)
        at += n
