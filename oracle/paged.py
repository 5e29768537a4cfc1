"""Plain fp64 oracle of the paged key / value cache, the attention over it and
the acceptance of drafts (test infrastructure only).

Written from the definitions in ``include/glinattn.h``; numpy, loops where they
are clearest.
"""
from __future__ import annotations

import math

import numpy as np

E_MIN, E_MAX = -100, 119
#: the non-negative finite e4m3 values, by code 0 .. 126
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)])


def positions(q_start, kv_len, r):
    """(row, position) pairs of request r's new tokens."""
    s0, s1 = int(q_start[r]), int(q_start[r + 1])
    return [(i, int(kv_len[r]) - (s1 - i)) for i in range(s0, s1)]


def scale_exponent(x):
    """Smallest e in [E_MIN, E_MAX] with every finite |x| <= 448 * 2^e (E_MAX: none has)."""
    x = np.abs(x[np.isfinite(x)])
    a = float(x.max()) if x.size else 0.0
    if a == 0.0:
        return E_MIN
    e = math.ceil(math.log2(a / 448.0))
    while a <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    while a > 448.0 * 2.0 ** e:
        e += 1
    return min(max(e, E_MIN), E_MAX)


def round_e4m3(y):
    """Nearest e4m3 value, ties to the even code; beyond 448 +-448; NaN stays."""
    a = np.abs(y)
    a = np.where(np.isnan(a), 0.0, np.minimum(a, 448.0))
    hi = np.minimum(np.searchsorted(E4M3, a, side="left"), 126)
    lo = np.maximum(hi - 1, 0)
    below, above = a - E4M3[lo], E4M3[hi] - a
    take_lo = (below < above) | ((below == above) & (lo % 2 == 0))
    v = np.copysign(np.where(take_lo, E4M3[lo], E4M3[hi]), y)
    return np.where(np.isnan(y), np.nan, v)


def quantise(x):
    """Rows x [..., d] as (e4m3 values, exponents)."""
    flat = x.reshape(-1, x.shape[-1])
    e = np.array([scale_exponent(r) for r in flat], np.int64)
    with np.errstate(over="ignore"):
        v = round_e4m3(flat * 2.0 ** -e[:, None].astype(np.float64))
    return v.reshape(x.shape), e.reshape(x.shape[:-1])


def attention(q, k_rows, v_rows, q_start, kv_len, scale):
    """q [N, H, d]; k_rows, v_rows: per request [kv_len, Hkv, d], all fp64.
    Returns (o, a): the outputs and sum_j p_j |v_j| (what a rounding of the
    weights is relative to); rows of no request are NaN."""
    N, H, d = q.shape
    o, a = np.full((N, H, d), np.nan), np.full((N, H, d), np.nan)
    for r in range(len(kv_len)):
        k, v = k_rows[r], v_rows[r]
        group = H // k.shape[1]
        for i, pos in positions(q_start, kv_len, r):
            if pos < 0:
                o[i], a[i] = 0.0, 0.0
                continue
            for h in range(H):
                s = scale * (k[:pos + 1, h // group] @ q[i, h])
                m = s.max()
                if m == -np.inf:
                    o[i, h], a[i, h] = 0.0, 0.0
                    continue
                p = np.exp(s - m)
                p /= p.sum()
                o[i, h] = p @ v[:pos + 1, h // group]
                a[i, h] = p @ np.abs(v[:pos + 1, h // group])
    return o, a


def accept_drafts(target, draft, tokens, uniforms, num_drafts=None):
    """target [R, D+1, V], draft [R, D, V] or None, all fp32 values; python
    integers for the cumulative draw.  Returns (accept [R], tokens [R, D+1])."""
    R, D1, V = target.shape
    f32 = np.float32
    out = np.full((R, D1), -1, np.int32)
    acc = np.zeros(R, np.int32)
    for r in range(R):
        n = D1 - 1 if num_drafts is None else int(num_drafts[r])
        a = 0
        while a < n:
            x = int(tokens[r, a])
            qx = f32(1) if draft is None else f32(draft[r, a, x])
            if not f32(f32(uniforms[r, a]) * qx) < f32(target[r, a, x]):
                break
            a += 1
        p = target[r, a].astype(f32)
        w = p.copy()
        if a < n and draft is not None:
            w = p - draft[r, a].astype(f32)
        elif a < n:
            w[int(tokens[r, a])] = 0

        def whole(x):
            x = np.where(np.isnan(x), f32(0), x)
            return [int(y) for y in (np.clip(x, f32(0), f32(1)).astype(np.float64) * 2.0 ** 40)]

        W = whole(w)
        if sum(W) == 0:
            W = whole(p)
        total = sum(W)
        t = min(int(float(f32(uniforms[r, D1 - 1])) * float(total)), total - 1)
        run, tok = 0, 0
        for tok in range(V):
            run += W[tok]
            if run > t:
                break
        acc[r] = a
        out[r, :a] = tokens[r, :a]
        out[r, a] = tok
    return acc, out
