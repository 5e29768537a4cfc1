"""Bounds of the layer parts' tests, from the arithmetic that the header states."""
import numpy as np
import torch

from oracle import paged as P

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative
EPS32 = 2.0 ** -24


def close(got, want, tol, what=""):
    """Every element within its bound; where the oracle has NaN the kernel has one too."""
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), what
    with np.errstate(invalid="ignore"):
        bad = ~nan & ~(np.abs(got - want) <= tol) & (got != want)
    if bad.any():
        i = tuple(int(v[0]) for v in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {i}: {got[i]} for {want[i]}, bound {np.broadcast_to(tol, want.shape)[i]}")


def check_pow2_codes(code, amax, rel):
    """Each code's exponent is the smallest whose 448 * 2^e holds the maximum, which the kernel knows to `rel`."""
    e = code.astype(np.int64) - 127
    top = 448.0 * 2.0 ** e.astype(np.float64)
    assert ((e >= P.E_MIN) & (e <= P.E_MAX)).all()
    assert ((amax * (1 - rel) <= top) | (e == P.E_MAX)).all()
    assert ((amax * (1 + rel) > top / 2) | (e == P.E_MIN)).all()


def check_e4m3(q, scale, want, err):
    """Stored e4m3 values q under `scale` (both as the kernel has them) against the numbers that they stand for: half a
    step of e4m3, 2^-4 of the value or 2^-10 in the subnormals, and what the number itself may be off (`err`)."""
    y = want / scale
    tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10) + err / scale * (1 + 2.0 ** -4)
    inside = np.clip(y, -448.0, 448.0)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(q), nan)
    bad = ~nan & ~(np.abs(q - inside) <= tol)
    assert not bad.any(), (q[bad][:4], inside[bad][:4], tol[bad][:4])
