"""The pieces of a hybrid stack together, as one serving step runs them: the residual norm, a state-space block
(short convolution, packed scan), the residual norm, a softmax layer (cache write with rotation, attention over the
cache).  Every call is checked against the oracle on the inputs that the step really gave it; then the same step from a
captured graph, on other streams, and as a speculative round (drafts verified, accepted, replayed)."""
import math

import numpy as np
import pytest
import torch

from gated_deltanet_02_gb300 import (glinattn_accept_drafts, glinattn_add_rms_norm, glinattn_kv_append_rope,
                                     glinattn_paged_attention, glinattn_selective_scan_packed, glinattn_short_conv)
from oracle import layer_parts as L
from oracle import paged as P

from helpers import f64
from layer_parts_helpers import EPS32, HALF, close
from paged_helpers import attention_tolerance, rows_of

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16
W, D, N, H, HKV, HD, PAGE = 64, 96, 16, 4, 2, 64, 16        # width, channels, states, heads


class Stack:
    """Weights, pools and cache of one state-space and one softmax layer for a few requests."""

    def __init__(self, seed, slots=8, pages=40):
        g = torch.Generator().manual_seed(seed)
        self.g = g
        f = lambda *s, k=1.0: (k * torch.randn(s, generator=g)).to(DEV)  # noqa: E731
        self.w1, self.w2 = 1 + f(W, k=0.1), 1 + f(W, k=0.1)
        self.inproj, self.xproj, self.dtproj = f(W, 2 * D, k=W ** -0.5), f(D, 6 + 2 * N, k=D ** -0.5), f(6, D, k=0.5)
        self.outproj, self.qkv = f(D, W, k=D ** -0.5), f(W, (H + 2 * HKV) * HD, k=W ** -0.5)
        self.conv_w, self.conv_b = f(D, 4, k=0.5), f(D, k=0.1)
        self.A, self.skip, self.bias = -torch.arange(1, N + 1, device=DEV).float() * torch.exp(f(D, N, k=0.1)), f(D), f(D) - 3
        self.inv = (10000.0 ** (-torch.arange(0, HD, 2, device=DEV, dtype=torch.float64) / HD)).float()
        self.conv_pool, self.pool = f(slots, 3, D).to(BF16), f(slots, D, N)
        self.k_cache, self.v_cache = f(pages, HKV, PAGE, HD).to(BF16), f(pages, HKV, PAGE, HD).to(BF16)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def batch(self, lengths, history):
        R, g = len(lengths), self.g
        kv = [a + b for a, b in zip(lengths, history)]
        n_page = [-(-t // PAGE) for t in kv]
        order = torch.randperm(self.k_cache.shape[0], generator=g).to(torch.int32)
        table = torch.zeros((R, max(n_page)), dtype=torch.int32)
        at = 0
        for r, n in enumerate(n_page):
            table[r, :n] = order[at:at + n]
            at += n
        i = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        n = sum(lengths)
        return dict(lengths=lengths, kv=kv, table=table.to(DEV), kv_len=i(kv), q_start=i([0] + list(np.cumsum(lengths))),
                    slots=torch.randperm(self.pool.shape[0], generator=g)[:R].to(torch.int32).to(DEV), resume=i([int(h > 0) for h in history]),
                    x=torch.randn((n, W), generator=g).to(BF16).to(DEV), res=torch.randn((n, W), generator=g).to(DEV))

    def step(self, b, max_len, stream=None, update=True, count=None):
        """One step; returns every intermediate."""
        o, kw = {}, dict(stream=stream)
        o["y1"], o["r1"], _ = glinattn_add_rms_norm(b["x"], self.w1, b["res"], **kw)
        o["xz"] = (o["y1"].float() @ self.inproj).to(BF16)
        packed = dict(resume=b["resume"], count=count, update_state=update, dev_status=self.status, **kw)
        o["conv"] = glinattn_short_conv(o["xz"][:, :D], self.conv_w, self.conv_b, self.conv_pool, b["slots"], b["q_start"], **packed)
        o["proj"] = (o["conv"].float() @ self.xproj).to(BF16)
        o["delta"] = (o["proj"][:, :6].float() @ self.dtproj).to(BF16)
        o["scan"] = glinattn_selective_scan_packed(o["conv"], o["delta"], o["proj"][:, 6:6 + N], o["proj"][:, 6 + N:], self.A, self.pool,
                                                   b["slots"], b["q_start"], max_q_len=max_len, z=o["xz"][:, D:], skip=self.skip,
                                                   delta_bias=self.bias, **packed)
        o["m"] = (o["scan"].float() @ self.outproj).to(BF16)
        o["y2"], o["r2"], _ = glinattn_add_rms_norm(o["m"], self.w2, o["r1"], **kw)
        o["qkv"] = (o["y2"].float() @ self.qkv).to(BF16).view(-1, H + 2 * HKV, HD)
        q, k, v = o["qkv"][:, :H], o["qkv"][:, H:H + HKV], o["qkv"][:, H + HKV:]
        where = (self.k_cache, self.v_cache, b["table"], b["kv_len"], b["q_start"])
        o["q"], _, _ = glinattn_kv_append_rope(q, k, v, self.inv, *where, dev_status=self.status, **kw)
        o["att"] = glinattn_paged_attention(o["q"], *where, max_q_len=max_len, dev_status=self.status, **kw)
        return o

    def state(self):
        return [t.clone() for t in (self.conv_pool, self.pool, self.k_cache, self.v_cache)]

    def restore(self, saved):
        for t, x in zip((self.conv_pool, self.pool, self.k_cache, self.v_cache), saved):
            t.copy_(x)


def verify(s, b, o, before):
    conv0, pool0, _, _ = before
    qs, slots, resume = b["q_start"].cpu().numpy(), b["slots"].cpu().numpy(), b["resume"].cpu().numpy()
    for y, r, x, res, w in (("y1", "r1", b["x"], b["res"], s.w1), ("y2", "r2", o["m"], o["r1"], s.w2)):
        want, h = L.add_rms_norm(f64(x), f64(res), f64(w), 1e-6)
        close(o[r], h, 2 * EPS32 * np.abs(h), r)
        close(o[y], want, (HALF[BF16] + 64 * EPS32) * np.abs(want), y)
    want, size, new = L.short_conv(f64(o["xz"][:, :D]), f64(s.conv_w), f64(s.conv_b), f64(conv0), slots, qs, resume)
    close(o["conv"], want, 6 * EPS32 * size + (8 * EPS32 + HALF[BF16]) * np.abs(want), "conv")
    close(s.conv_pool, new, 0.0, "conv pool")
    want, size, new, psize, decay = L.scan_packed(f64(o["conv"]), f64(o["delta"]), f64(o["proj"][:, 6:6 + N]), f64(o["proj"][:, 6 + N:]), f64(s.A),
                                                  f64(pool0), slots, qs, f64(o["xz"][:, D:]), f64(s.skip), f64(s.bias), resume)
    rel = (5 * min(max(b["lengths"]), 1 / (1 - decay)) + 8) * EPS32 * 2
    close(o["scan"], want, (rel + 32 * EPS32) * size + HALF[BF16] * np.abs(want), "scan")
    close(s.pool, new, np.where(new != f64(pool0), rel * psize, 0.0), "pool")
    pos = np.concatenate([np.arange(t - n, t) for n, t in zip(b["lengths"], b["kv"])])
    want, size = L.rotate(f64(o["qkv"][:, :H]), pos, f64(s.inv))
    close(o["q"], want, 8 * EPS32 * size + HALF[BF16] * np.abs(want), "q")
    c = dict(k_cache=s.k_cache.cpu(), v_cache=s.v_cache.cpu(), cache="bf16", table=b["table"].cpu(), page=PAGE, Hkv=HKV, d=HD,
             lengths=list(zip(b["lengths"], b["kv"])), q_start=b["q_start"].cpu(), kv_len=b["kv_len"].cpu())
    k, v = rows_of(c, "k"), rows_of(c, "v")
    want, size = L.rotate(f64(o["qkv"][:, H:H + HKV]), pos, f64(s.inv))
    close(np.concatenate([x[len(x) - n:] for x, n in zip(k, b["lengths"])]), want, 8 * EPS32 * size + HALF[BF16] * np.abs(want), "keys")
    assert np.array_equal(np.concatenate([x[len(x) - n:] for x, n in zip(v, b["lengths"])]), f64(o["qkv"][:, H + HKV:]))
    scale = 1 / math.sqrt(HD)
    q = f64(o["q"])
    want, mag = P.attention(q, k, v, c["q_start"], c["kv_len"], scale)
    assert (np.abs(f64(o["att"]) - want) <= attention_tolerance(c, q, want, mag, scale)).all()
    assert int(s.status.item()) == 0


STEPS = {"prompts": ([21, 1, 40], [0, 0, 0]), "mixed": ([5, 33, 1, 2], [9, 0, 30, 0]), "tokens": ([1] * 5, [3, 17, 0, 40, 15]), "drafts": ([4] * 4, [8, 1, 20, 33])}


@pytest.mark.parametrize("name", list(STEPS))
@pytest.mark.parametrize("how", ["eager", "graph", "stream"])
def test_step(name, how):
    s = Stack(3)
    b = s.batch(*STEPS[name])
    before, top = s.state(), max(b["lengths"])
    if how == "eager":
        o = s.step(b, top)
    elif how == "graph":
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            o = s.step(b, top)
        s.restore(before)
        graph.replay()
        torch.cuda.synchronize()
        first, after = {k: v.clone() for k, v in o.items()}, s.state()
        s.restore(before)
        graph.replay()                      # the same inputs and states again: the same bits
        torch.cuda.synchronize()
        assert all(torch.equal(first[k], o[k]) for k in o) and all(torch.equal(x, y) for x, y in zip(after, s.state()))
    else:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            o = s.step(b, top, stream=side)
        side.synchronize()
    torch.cuda.synchronize()
    verify(s, b, o, before)


def test_a_replayed_graph_serves_other_lengths():
    """Ranges, slots and lengths are read from device memory: the graph of one batch runs another of the same sizes."""
    s = Stack(5)
    a, b = s.batch([9, 30, 3], [0, 10, 4]), s.batch([20, 2, 20], [5, 0, 8])
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    before = s.state()
    with torch.cuda.graph(graph, stream=side):
        o = s.step(a, 30)
    s.restore(before)
    for k in ("kv_len", "q_start", "slots", "resume", "x", "res"):
        a[k].copy_(b[k])
    a["table"].zero_()
    a["table"][:, :b["table"].shape[1]].copy_(b["table"])
    graph.replay()
    torch.cuda.synchronize()
    verify(s, dict(b, table=a["table"]), o, before)


def test_two_speculative_rounds():
    """Drafts run without a new state, the accepted ones are replayed: the pools end as if only they had been run."""
    s, t = Stack(7), Stack(7)
    R, V, K = 4, 50, 3
    b = s.batch([K + 1] * R, [6, 1, 20, 33])
    g = torch.Generator().manual_seed(8)
    for _ in range(2):
        before = s.state()
        o = s.step(b, K + 1, update=False)
        assert torch.equal(s.conv_pool, before[0]) and torch.equal(s.pool, before[1])
        z = torch.randn((R, K + 1, V), generator=g) * 2
        target, draft = torch.softmax(z + 0.5 * torch.randn((R, K + 1, V), generator=g), -1).to(DEV), torch.softmax(z[:, :K], -1).to(DEV)
        tokens = torch.multinomial(draft.view(-1, V).cpu(), 1, generator=g).view(R, K).to(torch.int32).to(DEV)
        accept, _ = glinattn_accept_drafts(target, draft, tokens, torch.rand((R, K + 1), generator=g).to(DEV))
        count = accept + 1                     # the token before the drafts, and those accepted
        glinattn_short_conv(o["xz"][:, :D], s.conv_w, s.conv_b, s.conv_pool, b["slots"], b["q_start"], resume=b["resume"], count=count, outputs=False)
        glinattn_selective_scan_packed(o["conv"], o["delta"], o["proj"][:, 6:6 + N], o["proj"][:, 6 + N:], s.A, s.pool, b["slots"], b["q_start"],
                                       max_q_len=K + 1, delta_bias=s.bias, resume=b["resume"], count=count, outputs=False)
        # the other stack runs the accepted rows alone, one token a call
        n = count.cpu().tolist()
        for k in range(K + 1):
            on = [r for r in range(R) if n[r] > k]
            if not on:
                break
            rows, slots = torch.tensor([r * (K + 1) + k for r in on], device=DEV), b["slots"][on].contiguous()
            first = b["resume"][on].contiguous() if k == 0 else None
            pick = lambda name, a=None, e=None: o[name][rows][:, a:e]  # noqa: E731
            glinattn_short_conv(pick("xz", 0, D), t.conv_w, t.conv_b, t.conv_pool, slots, resume=first)
            glinattn_selective_scan_packed(pick("conv"), pick("delta"), pick("proj", 6, 6 + N), pick("proj", 6 + N), t.A, t.pool, slots,
                                           delta_bias=t.bias, resume=first)
        assert torch.equal(s.conv_pool, t.conv_pool)
        assert torch.equal(s.pool, t.pool)
        b["kv_len"].add_(1)
        b["resume"].fill_(1)
    assert int(s.status.item()) == 0


def test_two_streams_at_once():
    """Long requests on two streams, a workspace each, give what they give alone."""
    g = torch.Generator().manual_seed(9)
    calls = []
    for n in (5000, 3100):
        f = lambda *s: torch.randn(s, generator=g).to(BF16).to(DEV)  # noqa: E731
        calls.append((f(n, 256), f(n, 256), f(n, N), f(n, N), -torch.rand((256, N), generator=g).to(DEV) - 0.5))
    alone = [glinattn_selective_scan_packed(*c, q_start=torch.tensor([0, len(c[0])], dtype=torch.int32, device=DEV)) for c in calls]
    starts = [torch.tensor([0, len(c[0])], dtype=torch.int32, device=DEV) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        outs = [glinattn_selective_scan_packed(*c, q_start=q, stream=st) for c, q, st in zip(calls, starts, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, outs))
