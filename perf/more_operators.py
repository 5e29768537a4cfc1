"""Workloads of the pieces around a hybrid stack's sequence mixers, each in a plain form and as the framework's call.

A serving step of such a stack runs, beside the mixers themselves: the residual's addition with the norm in front of every
layer; in a state-space layer the short causal convolution and the selective scan with its step bias, skip and gate; in a
softmax layer the rotation of queries and keys on the way into the paged cache.  The token rows of all requests are packed one
behind another (``q_start``), states live in pools by slot.  ``own`` selects the side: False computes with elementary torch
operations in 32 bits (angles in 64), True calls the framework.
"""
import math
import random

import torch

own = False

NORM, CONV, SCAN, ROPE = "norm", "conv", "scan", "rope"
STEP, VERIFY, REPLAY = "step", "verify", "replay"    # new tokens; drafts without a new state; the accepted drafts' state alone
E_MIN, E_MAX = -100, 119                             # exponents of power-of-two scales
MOST_SCAN = 8191 * 4096 * 16                         # the largest listed cases, which no drawn one exceeds
MOST_ROWS = 15001 * 4096


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm(name, rows, width, act, res, out, group, pow2):
    """out: bf16, f32 or e4m3; with e4m3 a scale for every `group` elements (0: the row), a power of two or in 32 bits."""
    return dict(name=name, op=NORM, rows=rows, width=width, act=act, res=res, out=out, group=group, pow2=pow2)


def _conv(name, req, q, channels, taps, act, silu, bias, mode, resume, pad, mix):
    """req requests with q[0]..q[1] new tokens; resume: the share of them that continue from their slot."""
    return dict(name=name, op=CONV, req=req, q_lo=q[0], q_hi=q[1], channels=channels, taps=taps, act=act, silu=silu, bias=bias,
                mode=mode, resume=resume, pad=pad, mix=mix)


def _scan(name, req, q, channels, state, act, gate, mode, resume, pad, mix):
    return dict(name=name, op=SCAN, req=req, q_lo=q[0], q_hi=q[1], channels=channels, state=state, act=act, gate=gate, mode=mode,
                resume=resume, pad=pad, mix=mix)


def _rope(name, cache, req, q, ctx, heads, kv_heads, d, rot, pairs, page, mix):
    """req requests with q[0]..q[1] new tokens behind ctx[0]..ctx[1] cached ones; rot of d channels are rotated; pairs:
    neighbouring channels form a pair, else those half of rot apart."""
    return dict(name=name, op=ROPE, cache=cache, req=req, q_lo=q[0], q_hi=q[1], ctx_lo=ctx[0], ctx_hi=ctx[1], heads=heads,
                kv_heads=kv_heads, d=d, rot=rot, pairs=pairs, page=page, mix=mix)


def listed():
    return [
        # an interactive server's step: four tokens, the width of this repository's benchmark (16 heads of 128)
        _norm("norm decode 4", 4, 2048, "bf16", "bf16", "bf16", 0, False),
        # packed prompts in front of a matrix product in 8 bits, one scale a token
        _norm("norm prompts e4m3 rows", 15001, 4096, "bf16", "bf16", "e4m3", 0, False),
        # the residual stream kept in 32 bits, power-of-two scales for blocks of 32
        _norm("norm chunk e4m3 blocks", 2049, 8192, "bf16", "f32", "e4m3", 32, True),
        # the decode batch of this repository's scan benchmark
        _conv("conv decode 256", 256, (1, 1), 2048, 4, "bf16", True, True, STEP, 1.0, 0, 1),
        # prompts of a batch, some of them continued; channels are a slice of the in-projection's rows
        _conv("conv prompts packed", 8, (200, 4001), 4096, 4, "bf16", True, True, STEP, 0.5, 0, 2),
        # an odd number of channels in 32 bits, without bias and activation, rows of padding
        _conv("conv odd f32", 3, (50, 999), 1111, 3, "f32", False, False, STEP, 0.5, 5, 3),
        # the decode batch of the scan benchmark
        _scan("scan decode 256", 256, (1, 1), 2048, 16, "bf16", True, STEP, 1.0, 0, 4),
        # the drafts of a speculative round: outputs, no new state
        _scan("scan drafts 64x5", 64, (5, 5), 2048, 16, "bf16", True, VERIFY, 1.0, 0, 5),
        # prompts of a batch, some of them continued
        _scan("scan prompts packed", 8, (200, 4001), 2048, 16, "bf16", True, STEP, 0.5, 0, 6),
        # one long prompt
        _scan("scan prompt 8191", 1, (8191, 8191), 4096, 16, "bf16", True, STEP, 0.0, 0, 7),
        # one decode step, 256 requests with long histories
        _rope("rope decode 256", "bf16", 256, (1, 1), (1000, 6000), 16, 4, 128, 128, False, 16, 8),
        # whole prompts into a cache in 8 bits
        _rope("rope prompts e4m3", "e4m3", 8, (1500, 8000), (0, 300), 32, 8, 128, 128, False, 16, 9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    mix = rng.randrange(1 << 20)
    kind = rng.choice([NORM, CONV, SCAN, SCAN, ROPE])
    act = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if kind == NORM:
        width = _log(rng, 64, 16384)
        rows = _log(rng, 1, max(1, min(16384, MOST_ROWS // (width + 128))))
        out = rng.choice(["bf16", "f32", "e4m3", "e4m3"])
        group = rng.choice([0, 32, 64, 128]) if out == "e4m3" else 0
        if group or rng.random() < 0.5:                   # half the others have a width that no vector fits
            width += -width % (group or 8)
        c = _norm("", rows, width, act, rng.choice(["none", "bf16", "f32"]), out, group, out == "e4m3" and rng.random() < 0.5)
        return _drawn(c)
    if kind == ROPE:
        req = _log(rng, 1, 256)
        hi = _log(rng, 1, max(1, min(8000, 32000 // req)))
        d = rng.choice([64, 128, 128])
        kv_heads = rng.choice([1, 2, 4, 8])
        return _drawn(_rope("", rng.choice(["bf16", "e4m3"]), req, (rng.randint(0, hi), hi), (0, _log(rng, 1, 32768)),
                            kv_heads * rng.choice([1, 2, 3, 4]), kv_heads, d, rng.choice([d, d, d // 2, 16, 48]), rng.random() < 0.3,
                            rng.choice([16, 16, 32, 64, 128]), mix))
    mode = rng.choice([STEP, STEP, STEP, VERIFY, REPLAY])
    req = _log(rng, 1, 256)
    channels = _log(rng, 64, 8192 if kind == CONV else 6000)
    if rng.random() < 0.6:
        channels += -channels % 8
    state = rng.choice([8, 16, 16, 32])
    most = MOST_ROWS // channels if kind == CONV else min(8192, MOST_SCAN // (channels * state))
    hi = _log(rng, 1, max(1, min(8192, most // req))) if mode == STEP else rng.randint(1, max(1, min(8, most // req)))
    q = (rng.randint(0, hi), hi)
    resume, pad = rng.choice([0.0, 0.5, 1.0]) if mode == STEP else 1.0, rng.choice([0, 0, 7])
    if kind == CONV:
        return _drawn(_conv("", req, q, channels, rng.choice([2, 3, 4, 4]), act, rng.random() < 0.8, rng.random() < 0.8, mode, resume, pad, mix))
    return _drawn(_scan("", req, q, channels, state, act, rng.random() < 0.8, mode, resume, pad, mix))


def _drawn(c):
    return {k: v for k, v in c.items() if k != "name"}


def _lengths(c):
    """New tokens of every request: a matter of the case, so that its work is."""
    rng = random.Random(c["mix"])
    return [c["q_hi"]] + [rng.randint(c["q_lo"], c["q_hi"]) for _ in range(c["req"] - 1)]


def _cached(c):
    rng = random.Random(c["mix"] + 1)
    return [rng.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["req"])]


def _counts(c):
    """How many of a request's tokens are run: all, or the accepted drafts."""
    rng = random.Random(c["mix"] + 2)
    return [rng.randint(0, n) if c["mode"] == REPLAY else n for n in _lengths(c)]


def _resumed(c):
    rng = random.Random(c["mix"] + 3)
    return [int(rng.random() < c["resume"]) for _ in range(c["req"])]


TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    if c["op"] == NORM:
        act, width, rows = TYPES[c["act"]], c["width"], c["rows"]
        # a layer's output, and a residual stream with a few strong channels and tokens of different size
        s = dict(case=c, x=normal(rows, width, dtype=act), w=1.0 + 0.2 * normal(width), res=None, sum=None, scale=None)
        if c["res"] != "none":
            strong = 1.0 + 30.0 * (torch.rand(width, generator=g, device=dev) > 0.998)
            s["res"] = (normal(rows, width) * strong * normal(rows, 1).mul_(0.5).exp_()).to(TYPES[c["res"]])
            s["sum"] = torch.empty_like(s["res"])
        s["y"] = torch.empty((rows, width), dtype=TYPES[c["out"]], device=dev)
        if c["out"] == "e4m3":
            s["scale"] = torch.empty((rows, width // c["group"] if c["group"] else 1), dtype=torch.uint8 if c["pow2"] else torch.float32, device=dev)
            if c["pow2"]:
                s["scale"] = s["scale"].view(torch.float8_e8m0fnu)
        return s
    q = _lengths(c)
    s = dict(case=c, q_start=ints([0] + q).cumsum(0).to(torch.int32), n=sum(q), max_q=max(q))
    if c["op"] == ROPE:
        kv, page, d = [a + b for a, b in zip(q, _cached(c))], c["page"], c["d"]
        n_page = [-(-t // page) for t in kv]
        pages = sum(n_page) + max(1, sum(n_page) // 8)                      # the pool has pages of other requests too
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        table = torch.zeros((c["req"], max(1, max(n_page))), dtype=torch.int32, device=dev)
        first = ints([0] + n_page).cumsum(0)
        col = torch.arange(table.shape[1], device=dev)
        used = col[None] < ints(n_page)[:, None]
        s |= dict(table=torch.where(used, order[(first[:-1, None] + col).clamp(max=pages - 1)], table).contiguous(), kv_len=ints(kv))
        heads, kv_heads = c["heads"], c["kv_heads"]
        rows = normal(s["n"], heads + 2 * kv_heads, d, dtype=torch.bfloat16)   # the projection's rows: q, k and v are slices of them
        s |= dict(q=rows[:, :heads], k=rows[:, heads:heads + kv_heads], v=rows[:, heads + kv_heads:])
        s["q_out"] = torch.empty((s["n"], heads, d), dtype=torch.bfloat16, device=dev)
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, c["rot"], 2, device=dev, dtype=torch.float64) / c["rot"])).float()
        for name in ("k", "v"):
            s[name + "_cache"] = torch.zeros((pages, kv_heads, page, d), dtype=TYPES[c["cache"]], device=dev)
            s[name + "_scale"] = torch.full((pages, kv_heads, page), 127, dtype=torch.uint8, device=dev) if c["cache"] == "e4m3" else None
        return s
    act, ch, req = TYPES[c["act"]], c["channels"], c["req"]
    n = s["n"] + c["pad"]                                   # the last rows belong to no request
    slots = req + max(1, req // 4)                          # the pool has slots of other requests too
    s |= dict(slot_ids=torch.randperm(slots, generator=g, device=dev)[:req].to(torch.int32), resume=None, count=None)
    if c["resume"] < 1.0:
        s["resume"] = ints(_resumed(c))
    if c["mode"] == REPLAY:
        s["count"] = ints(_counts(c))
    s["y"] = torch.zeros((n, ch), dtype=act, device=dev)
    rows = normal(n, 2 * ch, dtype=act)                     # the in-projection's rows: the channels and their gates
    s |= dict(x=rows[:, :ch], z=rows[:, ch:])
    if c["op"] == CONV:
        s["w"] = normal(ch, c["taps"]) * 0.5
        s["bias"] = 0.1 * normal(ch) if c["bias"] else None
        s["pool"] = normal(slots, c["taps"] - 1, ch, dtype=act)
        return s
    if not c["gate"]:
        s["z"] = None
    rank = -(-ch // 16)
    proj = normal(n, rank + 2 * c["state"], dtype=act)      # the x-projection's rows: low-rank steps, then B and C
    s |= dict(B=proj[:, rank:rank + c["state"]], C=proj[:, rank + c["state"]:])
    s["x"] = (rows[:, :ch].float() * torch.sigmoid(rows[:, :ch].float())).to(act)       # a SiLU's outputs
    s["delta"] = normal(n, ch, dtype=act)
    step = torch.exp(torch.rand(ch, generator=g, device=dev) * math.log(100.0) + math.log(1e-3))   # steps of 0.001 .. 0.1
    s["delta_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -torch.arange(1, c["state"] + 1, device=dev, dtype=torch.float32) * torch.exp(0.1 * normal(ch, c["state"]))
    s["skip"] = 1.0 + 0.2 * normal(ch)
    s["pool"] = normal(slots, ch, c["state"])
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _pow2(code):
    """2^(code - 127) in 32 bits, exactly, for codes 1..254."""
    return (code.int() << 23).view(torch.float32)


def _code(amax):
    """Codes of the smallest power-of-two scales under which amax is at most 448."""
    f, e = torch.frexp(amax)
    e = torch.where(f <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX) + 127


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
        s["sum"].copy_(h)
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * s["w"]
    if c["out"] != "e4m3":
        s["y"].copy_(y)
        return _normed(s)
    y = y.view(c["rows"], s["scale"].shape[1], -1)
    amax = y.abs().amax(-1)
    if c["pow2"]:
        code = _code(amax)
        s["scale"].view(torch.uint8).copy_(code)
        y = y * _pow2(254 - code)[..., None]
    else:
        s["scale"].copy_((amax / 448.0).clamp_min(2.0 ** E_MIN))
        y = y / s["scale"][..., None]
    s["y"].copy_(y.clamp(-448.0, 448.0).view(c["rows"], -1))
    return _normed(s)


def _normed(s):
    return {k: s[k] for k in ("y", "sum", "scale") if s[k] is not None}


def _rows(s):
    """For every packed row: its request, its place in it, and whether it is run; for every request its number of rows run."""
    start, n = s["q_start"].long(), s["x"].shape[0]
    row = torch.arange(n, device=start.device)
    r = (torch.searchsorted(start, row, right=True) - 1).clamp(max=start.numel() - 2)
    i, length = row - start[r], start[1:] - start[:-1]
    count = length if s["count"] is None else s["count"].long()
    return row, r, i, i < count[r], start[:-1], count


def _history(s):
    """The requests' states at their start, in 32 bits."""
    h = s["pool"][s["slot_ids"].long()].float()
    return h if s["resume"] is None else h * (s["resume"] != 0).view(-1, 1, 1)


def _plain_conv(s):
    c, taps, n = s["case"], s["case"]["taps"], s["x"].shape[0]
    row, r, i, live, start, count = _rows(s)
    src = torch.cat([s["x"].float(), _history(s).reshape(-1, c["channels"])])
    back = torch.arange(taps - 1, -1, -1, device=row.device)
    if c["mode"] != REPLAY:
        at = i[:, None] - back
        y = (src[torch.where(at >= 0, row[:, None] - back, n + r[:, None] * (taps - 1) + taps - 1 + at)] * s["w"].T).sum(1)
        if s["bias"] is not None:
            y = y + s["bias"]
        if c["silu"]:
            y = y / (1.0 + torch.exp(-y))
        s["y"].copy_(torch.where(live[:, None], y, s["y"].float()))
    if c["mode"] != VERIFY:
        at = count[:, None] - back[:-1]
        new = src[torch.where(at >= 0, start[:, None] + at, n + torch.arange(c["req"], device=row.device)[:, None] * (taps - 1) + taps - 1 + at)]
        _keep(s, new, count)
    return _stepped(s)


def _keep(s, new, count):
    slots = s["slot_ids"].long()
    s["pool"][slots] = torch.where((count > 0).view(-1, 1, 1), new.to(s["pool"].dtype), s["pool"][slots])


def _stepped(s):
    mode = s["case"]["mode"]
    return ([s["y"]] if mode != REPLAY else []) + ([s["pool"]] if mode != VERIFY else [])


def _plain_scan(s):
    c = s["case"]
    row, r, i, live, start, count = _rows(s)
    x, d = s["x"].float(), s["delta"].float() + s["delta_bias"]
    dt = d.clamp_min(0.0) + torch.log1p(torch.exp(-d.abs()))
    a = torch.exp(dt[..., None] * s["A"])
    h = (dt * x)[..., None] * s["B"].float()[:, None]
    first = (i == 0) & live
    h[first] += a[first] * _history(s)[r[first]]
    a[first] = 0.0
    k = 1
    while k < s["max_q"]:                     # h_t = a_t h_{t-1} + b_t by doubling: after each step it reaches k rows back
        h, a = torch.cat([h[:k], torch.addcmul(h[k:], a[k:], h[:-k])]), torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    del a
    if c["mode"] != REPLAY:
        y = (h * s["C"].float()[:, None]).sum(-1) + s["skip"] * x
        if s["z"] is not None:
            z = s["z"].float()
            y = y * (z / (1.0 + torch.exp(-z)))
        s["y"].copy_(torch.where(live[:, None], y, s["y"].float()))
    if c["mode"] != VERIFY:
        _keep(s, h[(start + count - 1).clamp(0, max(0, s["n"] - 1))], count)
    return _stepped(s)


def _rotated(c, x, cos, sin):
    half, x = c["rot"] // 2, x.float()
    y = x.clone()
    u, v = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["pairs"] else (slice(0, half), slice(half, c["rot"]))
    y[..., u] = x[..., u] * cos - x[..., v] * sin
    y[..., v] = x[..., v] * cos + x[..., u] * sin
    return y


def _plain_rope(s):
    c, start = s["case"], s["q_start"].long()
    row = torch.arange(s["n"], device=start.device)
    r = torch.searchsorted(start, row, right=True) - 1
    pos = s["kv_len"].long()[r] - (start[r + 1] - row)
    angle = pos.double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    s["q_out"].copy_(_rotated(c, s["q"], cos, sin))
    page, at = s["table"].long()[r, pos // c["page"]], pos % c["page"]
    for name, x in (("k", _rotated(c, s["k"], cos, sin)), ("v", s["v"].float())):
        if c["cache"] == "e4m3":
            code = _code(x.abs().amax(-1))
            s[name + "_scale"][page, :, at] = code.to(torch.uint8)
            y = (x * _pow2(254 - code)[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            s[name + "_cache"].view(torch.uint8)[page, :, at] = y.view(torch.uint8)
        else:
            s[name + "_cache"][page, :, at] = x.to(torch.bfloat16)
    return _rotation(s)


def _rotation(s):
    out = {k: s[k] for k in ("q_out", "k_cache", "v_cache")}
    if s["k_scale"] is not None:                # codes of powers of two, as the numbers that they stand for
        out |= {k: s[k].view(torch.float8_e8m0fnu) for k in ("k_scale", "v_scale")}
    return out


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return _own(s, op)
    return {NORM: _plain_norm, CONV: _plain_conv, SCAN: _plain_scan, ROPE: _plain_rope}[op](s)


def _own(s, op):
    import gated_deltanet_02_gb300 as G
    c = s["case"]
    if op == NORM:
        G.glinattn_add_rms_norm(s["x"], s["w"], s["res"], eps=1e-6, group=c["group"], y=s["y"], residual_out=s["sum"], scale=s["scale"])
        return _normed(s)
    if op == ROPE:
        G.glinattn_kv_append_rope(s["q"], s["k"], s["v"], s["inv_freq"], s["k_cache"], s["v_cache"], s["table"], s["kv_len"], s["q_start"],
                                  interleaved=c["pairs"], q_out=s["q_out"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return _rotation(s)
    # single tokens need no ranges: request r is row r
    q_start = None if c["q_lo"] == c["q_hi"] == 1 and c["pad"] == 0 else s["q_start"]
    more = dict(resume=s["resume"], count=s["count"], update_state=c["mode"] != VERIFY, outputs=c["mode"] != REPLAY,
                y=s["y"] if c["mode"] != REPLAY else None)
    if op == CONV:
        G.glinattn_short_conv(s["x"], s["w"], s["bias"], s["pool"], s["slot_ids"], q_start, silu=c["silu"], **more)
    else:
        G.glinattn_selective_scan_packed(s["x"], s["delta"], s["B"], s["C"], s["A"], s["pool"], s["slot_ids"], q_start,
                                         max_q_len=s["max_q"], z=s["z"], skip=s["skip"], delta_bias=s["delta_bias"], **more)
    return _stepped(s)


# ---------------------------------------------------------------------------
# work, and the definition in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == NORM:
        e = dict(none=0, bf16=2, f32=4, e4m3=1)
        n = c["rows"] * c["width"]
        scales = c["rows"] * (c["width"] // c["group"] if c["group"] else 1) * (1 if c["pow2"] else 4) if c["out"] == "e4m3" else 0
        return dict(bytes=n * (e[c["act"]] + 2 * e[c["res"]] + e[c["out"]]) + scales + 4 * c["width"], flops=5 * n)
    n = sum(_lengths(c))
    if c["op"] == ROPE:
        row = c["kv_heads"] * (2 * c["d"] if c["cache"] == "bf16" else c["d"] + 1)
        return dict(bytes=max(1, n * (4 * c["heads"] * c["d"] + 4 * c["kv_heads"] * c["d"] + 2 * row)),
                    flops=3 * n * c["rot"] * (c["heads"] + c["kv_heads"]))
    n, e = max(1, sum(_counts(c))), 2 if c["act"] == "bf16" else 4
    begun = sum(k > 0 for k in _counts(c))
    reads = sum(f for f, k in zip(_resumed(c) if c["resume"] < 1.0 else [1] * c["req"], _counts(c)) if k > 0)
    states = reads + (begun if c["mode"] != VERIFY else 0)
    y = 1 if c["mode"] != REPLAY else 0
    if c["op"] == CONV:
        return dict(bytes=n * c["channels"] * e * (1 + y) + states * (c["taps"] - 1) * c["channels"] * e + 4 * c["channels"] * (c["taps"] + 1),
                    flops=n * c["channels"] * (2 * c["taps"] + 4) if y else n * c["channels"])
    streams = 2 + y + (y if c["gate"] else 0)
    return dict(bytes=n * c["channels"] * e * streams + n * c["state"] * e * (1 + y) + 4 * c["channels"] * (c["state"] + 2) +
                states * c["channels"] * c["state"] * 4, flops=7 * n * c["channels"] * c["state"])


def _exact_pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_exponent(a):
    """The smallest e with a <= 448 * 2^e, from the definition."""
    e = torch.full_like(a, E_MIN)
    for k in range(E_MIN, E_MAX):
        e = torch.where(a > 448.0 * 2.0 ** k, torch.full_like(e, k + 1.0), e)
    return e


def _exact_e4m3(y):
    """The nearest e4m3 value, ties to even: steps of 2^-9 at least, of an eighth of the leading power of two else."""
    step = _exact_pow2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3.0)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    s = prepare(case, seed)
    return {NORM: _exact_norm, CONV: _exact_conv, SCAN: _exact_scan, ROPE: _exact_rope}[case["op"]](case, s)


def _exact_norm(c, s):
    h = s["x"].double() + (s["res"].double() if s["res"] is not None else 0.0)
    y = s["w"].double() * h / torch.sqrt((h * h).sum(-1, keepdim=True) / c["width"] + 1e-6)
    out = dict(y=y, sum=h) if s["res"] is not None else dict(y=y)
    if c["out"] == "e4m3":
        blocks = y.unflatten(1, (s["scale"].shape[1], -1))
        top = blocks.abs().amax(-1)
        out["scale"] = _exact_pow2(_exact_exponent(top)) if c["pow2"] else torch.clamp(top / 448.0, min=2.0 ** E_MIN)
        out["y"] = _exact_e4m3(blocks / out["scale"][..., None]).flatten(1)
    return out


def _exact_conv(c, s):
    taps, at, y, pool = c["taps"], 0, s["y"].double(), s["pool"].double()
    slots, fresh = s["slot_ids"].tolist(), [not f for f in _resumed(c)] if c["resume"] < 1.0 else [False] * c["req"]
    for r, (length, run_) in enumerate(zip(_lengths(c), _counts(c))):
        past = pool[slots[r]].clone()
        if fresh[r]:
            past.zero_()
        line = torch.cat([past, s["x"][at:at + run_].double()])
        if run_:
            o = sum(line[j:j + run_] * s["w"][:, j].double() for j in range(taps))
            if s["bias"] is not None:
                o = o + s["bias"].double()
            y[at:at + run_] = o * torch.sigmoid(o) if c["silu"] else o
            pool[slots[r]] = line[run_:]
        at += length
    return ([y] if c["mode"] != REPLAY else []) + ([pool] if c["mode"] != VERIFY else [])


def _exact_scan(c, s):
    lengths, counts = _lengths(c), _counts(c)
    if c["req"] * max(counts) * c["channels"] * c["state"] > 4 * MOST_SCAN:
        return None
    y, pool, slots = s["y"].double(), s["pool"].double(), s["slot_ids"].long()
    dev = y.device
    h = pool[slots]
    if s["resume"] is not None:
        h = h * (s["resume"] != 0).double()[:, None, None]
    start, count = torch.tensor([sum(lengths[:r]) for r in range(c["req"])], device=dev), torch.tensor(counts, device=dev)
    A, skip, bias = s["A"].double(), s["skip"].double(), s["delta_bias"].double()
    for t in range(max(counts)):
        on = [r for r in range(c["req"]) if counts[r] > t] if c["req"] > 1 else [0]
        who = torch.tensor(on, device=dev)
        rows = start[who] + t
        x, dt = s["x"][rows].double(), torch.logaddexp(s["delta"][rows].double() + bias, torch.zeros((), dtype=torch.float64, device=dev))
        g = torch.exp(dt[:, :, None] * A) * h[who] + (dt * x)[:, :, None] * s["B"][rows].double()[:, None, :]
        h[who] = g
        o = torch.einsum("rdn,rn->rd", g, s["C"][rows].double()) + skip * x
        if s["z"] is not None:
            z = s["z"][rows].double()
            o = o * z * torch.sigmoid(z)
        y[rows] = o
    keep = count > 0
    pool[slots[keep]] = h[keep]
    return ([y] if c["mode"] != REPLAY else []) + ([pool] if c["mode"] != VERIFY else [])


def _exact_rope(c, s):
    lengths, cached = _lengths(c), _cached(c)
    dev, page, table = s["q"].device, c["page"], s["table"].cpu()
    pos = torch.cat([torch.arange(b, b + a) for a, b in zip(lengths, cached)])
    owner = torch.repeat_interleave(torch.arange(c["req"]), torch.tensor(lengths))
    pg, at = table[owner, pos // page].long().to(dev), (pos % page).to(dev)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=dev), pos.to(dev).double()[:, None] * s["inv_freq"].double())[:, None]
    half = c["rot"] // 2

    def rotate(x):
        x = x.double()
        u, v = (x[..., 0:c["rot"]:2], x[..., 1:c["rot"]:2]) if c["pairs"] else (x[..., :half], x[..., half:c["rot"]])
        w = torch.complex(u, v) * turn
        w = torch.stack([w.real, w.imag], -1 if c["pairs"] else -2).flatten(-2)
        return torch.cat([w, x[..., c["rot"]:]], -1)

    out = dict(q_out=rotate(s["q"]))
    for name, x in (("k", rotate(s["k"])), ("v", s["v"].double())):
        cache = s[name + "_cache"].double()
        if c["cache"] == "e4m3":
            scale = _exact_pow2(_exact_exponent(x.abs().amax(-1)))
            codes = _exact_pow2(s[name + "_scale"].double() - 127.0)
            codes[pg, :, at] = scale
            out[name + "_scale"], x = codes, _exact_e4m3(x / scale[..., None])
        cache[pg, :, at] = x
        out[name + "_cache"] = cache
    return out
