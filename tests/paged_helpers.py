"""Inputs, oracle views and tolerances of the paged-cache tests."""
import numpy as np
import torch

from oracle import paged as P

HALF_BF16, HALF_E4M3 = 2.0 ** -8, 2.0 ** -4  # half a step, relative


def paged_case(lengths, Hkv, d, page, cache, seed=0, spare=3, num_tok=None, first=0, fill=1.0):
    """lengths: (q_len, kv_len) per request.  Pool rows are all filled (other
    requests' values); pages are shuffled.  CPU tensors."""
    g = torch.Generator().manual_seed(seed)
    R = len(lengths)
    n_page = [-(-kv // page) for _, kv in lengths]
    pages = sum(n_page) + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((R, max(1, max(n_page, default=1))), -7, dtype=torch.int32)  # unread entries may be anything
    at = 0
    for r, n in enumerate(n_page):
        table[r, :n] = order[at:at + n]
        at += n
    start = np.concatenate([[first], first + np.cumsum([q for q, _ in lengths])]) if R else np.array([first])
    c = dict(table=table, kv_len=torch.tensor([kv for _, kv in lengths], dtype=torch.int32),
             q_start=torch.tensor(start, dtype=torch.int32), num_tok=int(start[-1]) if num_tok is None else num_tok,
             lengths=lengths, Hkv=Hkv, d=d, page=page, pages=pages, cache=cache, k_scale=None, v_scale=None)
    for name in ("k", "v"):
        x = (fill * torch.randn((pages, Hkv, page, d), generator=g)).to(torch.bfloat16)
        c[name + "_cache"] = x
        if cache == "e4m3":
            v, e = P.quantise(x.double().numpy())
            c[name + "_cache"] = torch.from_numpy(v).float().to(torch.float8_e4m3fn)
            c[name + "_scale"] = torch.from_numpy(e + 127).to(torch.uint8)
    return c


def rows_of(c, name):
    """Per request the values [kv_len, Hkv, d] that its cached rows stand for, fp64."""
    x = c[name + "_cache"].float().double().numpy()
    if c["cache"] == "e4m3":
        x = x * 2.0 ** (c[name + "_scale"].numpy().astype(np.float64) - 127)[..., None]
    out = []
    for r, (_, kv) in enumerate(c["lengths"]):
        t = np.arange(kv)
        out.append(x[c["table"][r].numpy()[t // c["page"]], :, t % c["page"]].reshape(kv, c["Hkv"], c["d"]))
    return out


def dev(c, device="cuda:0"):
    return {k: (v.to(device) if isinstance(v, torch.Tensor) else v) for k, v in c.items()}


def cache_args(g):
    return ((g["k_cache"], g["v_cache"], g["table"], g["kv_len"], g["q_start"]),
            dict(k_scale=g["k_scale"], v_scale=g["v_scale"]))


def attention_tolerance(c, q, o, a, scale):
    """Elementwise bound: the output's rounding (half a bf16 step of |o|), the
    weights' rounding (half a bf16 step of sum p |v|), and the error of the
    scores.  A score is an fp32 sum of d products, off by at most d 2^-24 times
    sum |q| |k|; a query split into two e4m3 parts (4 + 4 bits hold bf16's 8),
    scaled so that its largest element is at least 2^7, is off by half the
    smallest e4m3 step, 2^-10, or 2^-17 max |q|, at most: 2^-17 max |q| sum |k|.
    An error of ds in the scores moves
    an output by at most 2 ds sum p |v|."""
    qa = np.abs(q)
    ds = 0.0
    for r, k in enumerate(rows_of(c, "k")):
        if not len(k):
            continue
        group = q.shape[1] // c["Hkv"]
        for i, pos in P.positions(c["q_start"], c["kv_len"], r):
            if pos < 0:
                continue
            for h in range(q.shape[1]):
                ka = np.abs(k[:pos + 1, h // group])
                ds = max(ds, float((ka @ qa[i, h]).max()) * c["d"] * 2.0 ** -24 +
                         float(ka.sum(-1).max()) * float(qa[i, h].max()) * 2.0 ** -17)
    ds = ds * scale + 2.0 ** -20  # and the exponential's own error
    return HALF_BF16 * np.abs(o) + (HALF_BF16 + 2 * ds) * a + 1e-30
