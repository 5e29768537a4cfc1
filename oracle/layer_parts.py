"""Plain fp64 oracle of the pieces around the sequence mixers: the residual norm,
the packed short convolution, the packed selective scan, the position rotation
(test infrastructure only).

Written from the definitions in ``include/glinattn.h``; numpy, loops where they
are clearest.  Where a tolerance needs it a function also returns the size of
what was added up.
"""
from __future__ import annotations

import numpy as np

from .selective_scan import softplus


def add_rms_norm(x, residual, weight, eps):
    """(y, h) of rows x [rows, width]; residual or weight may be None."""
    h = x if residual is None else x + residual
    with np.errstate(invalid="ignore"):
        y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return (y if weight is None else y * weight), h


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))


def ranges(q_start, num_tok, count=None, max_len=None):
    """(first row, rows, rows that are run) per request, None for one that is out of bounds."""
    out = []
    for r in range(len(q_start) - 1):
        s0, s1 = int(q_start[r]), int(q_start[r + 1])
        run = s1 - s0 if count is None else int(count[r])
        good = 0 <= s0 <= s1 <= num_tok and 0 <= run <= s1 - s0 and (max_len is None or s1 - s0 <= max_len)
        out.append((s0, s1 - s0, run) if good else None)
    return out


def short_conv(x, w, bias, pool, slots, q_start, resume=None, count=None, act=True):
    """x [n, C], w [C, W], pool [P, W-1, C] or None.  Returns (y, size, pool'):
    rows that are not run are NaN; size is sum |w x| + |bias| under the activation."""
    n, C = x.shape
    W = w.shape[1]
    y, size = np.full((n, C), np.nan), np.full((n, C), np.nan)
    new = None if pool is None else pool.copy()
    for r, rng in enumerate(ranges(q_start, n, count)):
        if rng is None or (pool is not None and not 0 <= slots[r] < len(pool)):
            continue
        s0, _, run = rng
        past = np.zeros((W - 1, C))
        if pool is not None and (resume is None or resume[r]):
            past = pool[slots[r]]
        line = np.concatenate([past, x[s0:s0 + run]])
        if run == 0:
            continue
        b = 0.0 if bias is None else bias
        o = sum(line[j:j + run] * w[:, j] for j in range(W)) + b
        y[s0:s0 + run] = silu(o) if act else o
        size[s0:s0 + run] = sum(np.abs(line[j:j + run] * w[:, j]) for j in range(W)) + np.abs(b)
        if new is not None:
            new[slots[r]] = line[run:]
    return y, size, new


def scan_packed(x, delta, Bm, Cm, A, pool, slots, q_start, z=None, skip=None, bias=None, resume=None, count=None, max_len=None):
    """Returns (y, y_size, pool', pool_size, decay): rows that are not run are NaN, the
    sizes are those of the sums of absolute values, decay the largest exp(dt A)."""
    n, D = x.shape
    N = A.shape[1]
    y, ysize = np.full((n, D), np.nan), np.full((n, D), np.nan)
    new = None if pool is None else pool.copy()
    psize = None if pool is None else np.abs(pool)
    decay = 0.0
    for r, rng in enumerate(ranges(q_start, n, count, max_len)):
        if rng is None or (pool is not None and not 0 <= slots[r] < len(pool)):
            continue
        s0, _, run = rng
        h = np.zeros((D, N))
        if pool is not None and (resume is None or resume[r]):
            h = pool[slots[r]].copy()
        a = np.abs(h)
        for t in range(s0, s0 + run):
            dt = softplus(delta[t] + (0.0 if bias is None else bias))
            E = np.exp(dt[:, None] * A)
            decay = max(decay, float(E.max()))
            b = (dt * x[t])[:, None] * Bm[t]
            h, a = E * h + b, E * a + np.abs(b)
            o, g = (h * Cm[t]).sum(-1), (a * np.abs(Cm[t])).sum(-1)
            if skip is not None:
                o, g = o + skip * x[t], g + np.abs(skip * x[t])
            if z is not None:
                o, g = o * silu(z[t]), g * np.abs(silu(z[t]))
            y[t], ysize[t] = o, g
        if run and new is not None:
            new[slots[r]], psize[slots[r]] = h, a
    return y, ysize, new, psize, decay


def rotate(x, pos, inv_freq, interleaved=False, scale=1.0):
    """x [n, heads, d] at positions pos [n].  Returns (rotated, size): size is the sum of the absolute products."""
    half, rot = len(inv_freq), 2 * len(inv_freq)
    # the angle modulo a turn in extended precision
    turn = np.asarray(pos, np.longdouble)[:, None] * np.asarray(inv_freq, np.longdouble)
    ang = np.asarray(turn - np.floor(turn / (2 * PI)) * (2 * PI), np.float64)
    c, s = scale * np.cos(ang)[:, None], scale * np.sin(ang)[:, None]
    u, v = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, half), slice(half, rot))
    y, size = x.copy(), np.abs(x)
    y[..., u], y[..., v] = x[..., u] * c - x[..., v] * s, x[..., v] * c + x[..., u] * s
    size[..., u] = size[..., v] = abs(scale) * (np.abs(x[..., u]) + np.abs(x[..., v]))
    return y, size


#: pi in extended precision, from its decimal digits
PI = np.longdouble("3.14159265358979323846264338327950288")
