"""Workloads of the softmax-attention and draft-acceptance operators, each in a plain form and as the framework's call.

The cases stand for one serving step of a hybrid stack's softmax layers (writing the new tokens' keys and values into the
paged cache, reading them back, attention over the cache) and for the acceptance of drafted tokens.  ``own`` selects the side:
False computes with elementary torch operations in 32 bits, True calls the framework.
"""
import math
import random

import torch

own = False

ATTENTION, APPEND, GATHER, ACCEPT = "attention", "append", "gather", "accept"
E_MIN, E_MAX = -100, 119      # exponents of the cache's power-of-two scales
WEIGHT = 2.0 ** 40            # probabilities become whole numbers of this size


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _att(name, cache, req, q, ctx, heads, kv_heads, d, page, mix):
    """req requests with q[0]..q[1] new tokens after ctx[0]..ctx[1] cached ones."""
    return dict(name=name, op=ATTENTION, cache=cache, req=req, q_lo=q[0], q_hi=q[1], ctx_lo=ctx[0], ctx_hi=ctx[1],
                heads=heads, kv_heads=kv_heads, d=d, page=page, mix=mix)


def _kv(name, op, cache, req, q, ctx, kv_heads, d, page, mix):
    return dict(name=name, op=op, cache=cache, req=req, q_lo=q[0], q_hi=q[1], ctx_lo=ctx[0], ctx_hi=ctx[1],
                kv_heads=kv_heads, d=d, page=page, mix=mix)


def _acc(name, req, drafts, vocab, point, mix):
    return dict(name=name, op=ACCEPT, req=req, drafts=drafts, vocab=vocab, point=point, mix=mix)


def listed():
    return [
        # an interactive server's step: four requests with short histories, one token each
        _att("attention decode 4", "bf16", 4, (1, 1), (0, 900), 16, 4, 128, 16, 1),
        # the decode batch of this repository's benchmark (256 requests, 16 heads of 128)
        _att("attention decode 256", "bf16", 256, (1, 1), (1000, 6000), 16, 4, 128, 16, 2),
        # its long-context round: 64 requests check 4 drafts each after some 32k tokens, cache in 8 bits
        _att("attention drafts 64x5 e4m3", "e4m3", 64, (5, 5), (31000, 32768), 32, 4, 128, 64, 3),
        # prompts of a batch packed one behind another, none of them cached before
        _att("attention prompts packed", "bf16", 8, (200, 4001), (0, 0), 16, 4, 128, 16, 4),
        # one long prompt, every head with its own keys, head size 64
        _att("attention prompt 8191 d64", "bf16", 1, (8191, 8191), (0, 0), 8, 8, 64, 32, 5),
        # a later piece of a long prompt over the pieces before it, cache in 8 bits
        _att("attention chunk 4096 e4m3", "e4m3", 1, (4096, 4096), (12288, 12288), 32, 8, 128, 64, 6),
        # one decode step's keys and values, 256 requests
        _kv("append decode 256 e4m3", APPEND, "e4m3", 256, (1, 1), (100, 1000), 4, 128, 16, 7),
        # whole prompts
        _kv("append prompts e4m3", APPEND, "e4m3", 8, (1500, 8000), (0, 300), 8, 128, 16, 8),
        # a short prefix handed to another engine
        _kv("gather prefixes bf16", GATHER, "bf16", 5, (33, 700), (0, 50), 4, 64, 16, 9),
        # long prefixes handed over
        _kv("gather long e4m3", GATHER, "e4m3", 4, (20000, 32768), (0, 0), 4, 128, 64, 10),
        # one request, 4 drafts
        _acc("accept 1x4", 1, 4, 100003, False, 11),
        # the whole decode batch
        _acc("accept 256x4", 256, 4, 160000, False, 12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    mix = rng.randrange(1 << 20)
    kind = rng.choice([ATTENTION, ATTENTION, ATTENTION, APPEND, GATHER, ACCEPT])
    cache = rng.choice(["bf16", "e4m3"])
    d, page = rng.choice([64, 128, 128]), rng.choice([16, 16, 32, 64, 128])
    if kind == ACCEPT:
        return _drawn(_acc("", _log(rng, 1, 256), rng.randint(0, 8), _log(rng, 1000, 160000), rng.random() < 0.3, mix))
    if kind in (APPEND, GATHER):
        req = _log(rng, 1, 256)
        top = max(1, min(32768, 131072 // req))
        hi = _log(rng, 1, top)
        return _drawn(_kv("", kind, cache, req, (rng.randint(0, hi), hi), (0, rng.randint(0, 1000)), rng.choice([1, 2, 4, 8]), d,
                          page, mix))
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    if rng.random() < 0.5:            # decode, with or without drafts
        req = _log(rng, 1, 256)
        ctx = _log(rng, 1, min(32768, 4000000 // (req * kv_heads)))
        q = rng.randint(1, 6)
        return _drawn(_att("", cache, req, (rng.randint(1, q), q), (rng.randint(0, ctx), ctx), kv_heads * group, kv_heads, d, page,
                           mix))
    req = _log(rng, 1, 16)            # prompts and pieces of prompts
    hi = _log(rng, 10, min(8000, 16000 // req))
    ctx = rng.choice([0, _log(rng, 1, 16000 // req)])
    while req * kv_heads * group * hi * (hi + ctx) > 1.8e9:     # at most the largest listed one's scores
        hi, ctx = max(1, hi // 2), ctx // 2
    return _drawn(_att("", cache, req, (rng.randint(0, hi), hi), (rng.randint(0, ctx), ctx), kv_heads * group, kv_heads, d, page, mix))


def _drawn(c):
    return {k: v for k, v in c.items() if k != "name"}


def _lengths(c):
    """New tokens and cache length of every request: a matter of the case, so that its work is."""
    rng = random.Random(c["mix"])
    q = [c["q_hi"]] + [rng.randint(c["q_lo"], c["q_hi"]) for _ in range(c["req"] - 1)]
    return q, [n + rng.randint(c["ctx_lo"], c["ctx_hi"]) for n in q]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _pow2(code):
    """2^(code - 127) in 32 bits, exactly, for codes 1..254."""
    return (code.int() << 23).view(torch.float32)


def _quantise(x):
    """Rows of x [..., d] as e4m3 values and the codes of their power-of-two scales."""
    x = x.float()
    a = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
    f, e = torch.frexp(a)
    e = torch.where(f <= 0.875, e - 9, e - 8)
    e = torch.where(a > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    y = (x * _pow2(127 - e)[..., None]).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _values(cache, scale):
    """The numbers that the cache's rows stand for, in 32 bits."""
    if scale is None:
        return cache.float()
    return cache.float() * _pow2(scale)[..., None]


def _paged(c, g, dev):
    q, kv = _lengths(c)
    page, n_page = c["page"], [-(-t // c["page"]) for t in kv]
    total = sum(n_page)
    pages = total + max(1, total // 8)                      # the pool has pages of other requests too
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((c["req"], max(1, max(n_page))), 0, dtype=torch.int32, device=dev)
    start = torch.tensor([0] + n_page, device=dev).cumsum(0)
    col = torch.arange(table.shape[1], device=dev)
    used = col[None] < torch.tensor(n_page, device=dev)[:, None]
    table = torch.where(used, order[(start[:-1, None] + col).clamp(max=pages - 1)], table)
    s = dict(table=table.contiguous(), kv_len=torch.tensor(kv, dtype=torch.int32, device=dev),
             q_start=torch.tensor([0] + q, device=dev).cumsum(0).to(torch.int32), n=sum(q), max_q=max(q), pages=pages)
    for name in ("k", "v"):
        rows = torch.randn((pages, c["kv_heads"], page, c["d"]), generator=g, device=dev, dtype=torch.bfloat16)
        s[name + "_cache"], s[name + "_scale"] = rows, None
        if c["cache"] == "e4m3":
            s[name + "_cache"], s[name + "_scale"] = _quantise(rows)
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    c = case
    if c["op"] == ACCEPT:
        r, n, v = c["req"], c["drafts"], c["vocab"]
        z = torch.randn((r, n + 1, v), generator=g, device=dev) * 2.5
        target = torch.softmax(z + 0.6 * torch.randn((r, n + 1, v), generator=g, device=dev), -1)
        draft = torch.softmax(z[:, :n], -1)
        if c["point"]:                                      # drafts picked greedily: no draft distribution
            tokens = draft.argmax(-1).to(torch.int32)
        else:
            noise = torch.rand((r, n, v), generator=g, device=dev).clamp_min_(1e-20).log_().neg_()
            tokens = (draft / noise).argmax(-1).to(torch.int32)
        limit = random.Random(c["mix"])
        count = torch.tensor([limit.randint(n // 2, n) for _ in range(r)], dtype=torch.int32, device=dev)
        return dict(case=c, target=target, draft=None if c["point"] else draft, tokens=tokens, count=count,
                    u=torch.rand((r, n + 1), generator=g, device=dev))
    s = _paged(c, g, dev)
    s["case"] = c
    if c["op"] == ATTENTION:
        s["q"] = (2.0 * torch.randn((s["n"], c["heads"], c["d"]), generator=g, device=dev)).to(torch.bfloat16)
        s["o"] = torch.empty_like(s["q"])
    elif c["op"] == APPEND:
        for name in ("k", "v"):
            size = torch.randn((s["n"], c["kv_heads"], 1), generator=g, device=dev).exp()   # rows of different magnitude
            s[name] = (size * torch.randn((s["n"], c["kv_heads"], c["d"]), generator=g, device=dev)).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _where(s):
    """Page and row in the page of every new token's position."""
    c, start = s["case"], s["q_start"].long()
    row = torch.arange(s["n"], device=start.device)
    r = torch.searchsorted(start, row, right=True) - 1
    pos = s["kv_len"].long()[r] - (start[r + 1] - row)
    return s["table"].long()[r, pos // c["page"]], pos % c["page"]


def _plain_append(s):
    page, row = _where(s)
    for name in ("k", "v"):
        x = s[name]
        if s["case"]["cache"] == "e4m3":
            x, code = _quantise(x)
            s[name + "_scale"][page, :, row] = code
            s[name + "_cache"].view(torch.uint8)[page, :, row] = x.view(torch.uint8)
        else:
            s[name + "_cache"][page, :, row] = x
    return _cache(s)


def _cache(s):
    return {k: s[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale") if s[k] is not None}


def _plain_gather(s):
    page, row = _where(s)
    out = []
    for name in ("k", "v"):
        x, code = s[name + "_cache"], s[name + "_scale"]
        x = x.view(torch.uint8)[page, :, row].view(x.dtype) if code is not None else x[page, :, row]
        out.append(_values(x, None if code is None else code[page, :, row]).to(torch.bfloat16))
    return out


def _rows(s, name, most):
    """Every request's keys (or values), padded to the longest: [req, kv_heads, most, d] in 32 bits."""
    c, pages = s["case"], s["table"].long()
    x, code = s[name + "_cache"], s[name + "_scale"]
    x = x.view(torch.uint8)[pages].view(x.dtype) if code is not None else x[pages]
    x = _values(x, None if code is None else code[pages])
    return x.transpose(1, 2).reshape(c["req"], c["kv_heads"], -1, c["d"])[:, :, :most]


def _plain_attention(s):
    c, start = s["case"], s["q_start"].long()
    dev, group, length = start.device, c["heads"] // c["kv_heads"], start[1:] - start[:-1]
    q_len, kv_len = _lengths(c)
    most_q, most_k = max(1, max(q_len)), max(1, max(kv_len))
    row = torch.arange(s["n"], device=dev)
    r = torch.searchsorted(start, row, right=True) - 1
    q = torch.zeros((c["req"], most_q, c["heads"], c["d"]), device=dev)
    q[r, row - start[r]] = s["q"].float() * (1.0 / math.sqrt(c["d"]))
    q = q.view(c["req"], most_q, c["kv_heads"], group, c["d"]).transpose(1, 2).reshape(c["req"], c["kv_heads"], most_q * group, c["d"])
    p = q @ _rows(s, "k", most_k).transpose(-1, -2)
    last = (s["kv_len"].long() - length)[:, None] + torch.arange(most_q, device=dev)            # the last key that a token sees
    seen = torch.arange(p.shape[-1], device=dev) <= last.repeat_interleave(group, 1)[:, None, :, None]
    p.masked_fill_(~seen, -math.inf)
    m = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ _rows(s, "v", most_k)) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(c["req"], c["kv_heads"], most_q, group, c["d"]).transpose(1, 2).reshape(c["req"], most_q, c["heads"], c["d"])
    s["o"].copy_(o[r, row - start[r]])
    return s["o"]


def _plain_accept(s):
    target, draft, tokens, u = s["target"], s["draft"], s["tokens"].long(), s["u"]
    r, n, v = target.shape[0], tokens.shape[1], target.shape[2]
    dev, req = target.device, torch.arange(target.shape[0], device=target.device)
    count = s["count"].long()
    at = tokens[..., None]
    p_at = target[:, :n].gather(-1, at)[..., 0]
    q_at = torch.ones_like(p_at) if draft is None else draft.gather(-1, at)[..., 0]
    good = (u[:, :n] * q_at < p_at) & (torch.arange(n, device=dev) < count[:, None])
    a = good.long().cumprod(-1).sum(-1)
    p, rejected = target[req, a], a < count
    w = p
    if n:
        near = a.clamp(max=n - 1)
        if draft is None:
            w = p.clone()
            w[req, tokens[req, near]] = torch.where(rejected, torch.zeros_like(u[:, 0]), w[req, tokens[req, near]])
        else:
            w = torch.where(rejected[:, None], p - draft[req, near], p)
    whole = (w.clamp(0.0, 1.0) * WEIGHT).long()
    none = whole.sum(-1, keepdim=True) == 0                 # nothing left of the target: sample the target itself
    whole = torch.where(none, (p.clamp(0.0, 1.0) * WEIGHT).long(), whole)
    upto = whole.cumsum(-1)
    total = upto[:, -1]
    t = torch.minimum((u[:, n].double() * total.double()).long(), total - 1)
    last = (upto <= t[:, None]).sum(-1)
    out = torch.full((r, n + 1), -1, dtype=torch.int32, device=dev)
    col = torch.arange(n, device=dev)
    out[:, :n] = torch.where(col < a[:, None], tokens, -1).to(torch.int32)
    out[req, a] = last.to(torch.int32)
    return a.to(torch.int32), out


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return _own(s, op)
    return {ATTENTION: _plain_attention, APPEND: _plain_append, GATHER: _plain_gather, ACCEPT: _plain_accept}[op](s)


def _own(s, op):
    import gated_deltanet_02_gb300 as G
    if op == ACCEPT:
        return G.glinattn_accept_drafts(s["target"], s["draft"], s["tokens"], s["u"], num_drafts=s["count"])
    where = (s["table"], s["kv_len"], s["q_start"])
    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
    if op == APPEND:
        G.glinattn_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], *where, **scales)
        return _cache(s)
    if op == GATHER:
        return list(G.glinattn_kv_gather(s["k_cache"], s["v_cache"], *where, num_tok=s["n"], **scales))
    return G.glinattn_paged_attention(s["q"], s["k_cache"], s["v_cache"], *where, max_q_len=s["max_q"], o=s["o"], **scales)


# ---------------------------------------------------------------------------
# work, and the definition in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == ACCEPT:
        # the target's row that is sampled, half the time the draft's (after a rejection), a few numbers for each draft
        row = 4 * c["vocab"]
        return dict(bytes=int(c["req"] * (row * (1.0 if c["point"] or not c["drafts"] else 1.5) + 24 * (c["drafts"] + 1))),
                    flops=3 * c["req"] * c["vocab"])
    q, kv = _lengths(c)
    n, size, extra = sum(q), (2 if c["cache"] == "bf16" else 1), (0 if c["cache"] == "bf16" else 1)
    row = c["kv_heads"] * (c["d"] * size + extra)
    if c["op"] in (APPEND, GATHER):
        return dict(bytes=max(1, 2 * n * (row + 2 * c["kv_heads"] * c["d"])), flops=4 * n * c["kv_heads"] * c["d"])
    seen = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(q, kv))
    return dict(bytes=4 * n * c["heads"] * c["d"] + 2 * sum(kv) * row, flops=4 * c["heads"] * c["d"] * seen)


def _exact_pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_code(x):
    """Scale exponents from the definition: the smallest e with max |x| <= 448 * 2^e."""
    a = x.abs().amax(-1)
    e = torch.full_like(a, E_MIN)
    for k in range(E_MIN, E_MAX):
        e = torch.where(a > 448.0 * 2.0 ** k, torch.full_like(e, k + 1.0), e)
    return e


def _exact_e4m3(y):
    """The nearest e4m3 value, ties to even: steps of 2^-9 at least, of an eighth of the leading power of two else."""
    step = _exact_pow2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3.0)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == ACCEPT:
        return None                    # whole numbers only
    q_len, kv_len = _lengths(c)
    start = [0]
    for n in q_len:
        start.append(start[-1] + n)
    dev, table, page = s["table"].device, s["table"].cpu(), c["page"]

    def cells(r, first, last):
        pos = torch.arange(first, last)
        return table[r].long()[pos // page].to(dev), (pos % page).to(dev)

    if c["op"] == APPEND:
        out = {}
        for name in ("k", "v"):
            cache = s[name + "_cache"].double()
            for r in range(c["req"]):
                pg, row = cells(r, kv_len[r] - q_len[r], kv_len[r])
                x = s[name][start[r]:start[r + 1]].double()
                if c["cache"] == "e4m3":
                    x = _exact_e4m3(x * _exact_pow2(-_exact_code(x))[..., None])
                cache[pg, :, row] = x
            out[name + "_cache"] = cache
            if c["cache"] == "e4m3":
                out[name + "_scale"] = None
        return out

    def read(name, pg, row):
        x = s[name + "_cache"]
        x = (x.view(torch.uint8)[pg, :, row].view(x.dtype) if c["cache"] == "e4m3" else x[pg, :, row]).double()
        if c["cache"] == "e4m3":
            x = x * _exact_pow2(s[name + "_scale"][pg, :, row].double() - 127.0)[..., None]
        return x

    if c["op"] == GATHER:
        return [torch.cat([read(name, *cells(r, kv_len[r] - q_len[r], kv_len[r])) for r in range(c["req"])]) for name in ("k", "v")]
    group = c["heads"] // c["kv_heads"]
    if 4.0 * c["heads"] * c["d"] * sum(a * b for a, b in zip(q_len, kv_len)) > 8e12:
        return None
    out = torch.zeros((s["n"], c["heads"], c["d"]), dtype=torch.float64, device=dev)
    for r in range(c["req"]):
        if q_len[r] == 0 or kv_len[r] == 0:
            continue
        pg, row = cells(r, 0, kv_len[r])
        k, v = read("k", pg, row), read("v", pg, row)
        qr = s["q"][start[r]:start[r + 1]].double()
        hidden = torch.arange(kv_len[r], device=dev)[None] > (torch.arange(q_len[r], device=dev) + kv_len[r] - q_len[r])[:, None]
        for h in range(c["heads"]):
            z = (qr[:, h] @ k[:, h // group].T) / math.sqrt(c["d"])
            out[start[r]:start[r + 1], h] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ v[:, h // group]
    return out
