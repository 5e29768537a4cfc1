"""Draft acceptance over rows of many steps a warp, against whole-number sums."""
import numpy as np
import pytest
import torch

from gated_deltanet_02_gb300 import glinattn_accept_drafts

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _run(target, draft, drafted, u):
    a, t = glinattn_accept_drafts(target.to(DEV), None if draft is None else draft.to(DEV), drafted.to(DEV), u.to(DEV))
    return a.cpu().numpy(), t.cpu().numpy()


def _whole(x):
    x = np.where(np.isnan(x), np.float32(0), x)
    return (np.clip(x, 0, 1).astype(np.float64) * 2.0 ** 40).astype(np.int64)


def _draw(w, u):
    """The token of weights w (whole numbers, sum below 2^63) for a uniform number."""
    upto = np.cumsum(w)
    total = int(upto[-1])
    t = min(int(float(np.float32(u)) * float(total)), total - 1)
    return int(np.searchsorted(upto, t, side="right"))


@pytest.mark.parametrize("V", [24511, 24576, 24577, 100003, 160000, 200003, (1 << 22) - 1, 1 << 22])
def test_large_vocabularies(V):
    """Rows of several full steps a warp: the row itself, a residual, and the sums' largest size."""
    R = 3 if V > 1 << 20 else 8
    g = torch.Generator().manual_seed(V)
    target = torch.softmax(2.5 * torch.randn((R, 1, V), generator=g), -1)
    target[1] = 1.0 - torch.rand((1, V), generator=g) * 2.0 ** -20      # weights next to one: sums up to 2^62
    target[2] = 0.0
    target[2, 0, ::997] = 2.0 ** -30
    u = torch.rand((R, 1), generator=g)
    u[1], u[2] = 1.0 - 2.0 ** -24, 0.0
    none = torch.zeros((R, 0), dtype=torch.int32)
    want = [_draw(_whole(target[r, 0].numpy()), u[r, 0]) for r in range(R)]
    a, t = _run(target, None, none, u)
    assert (a == 0).all() and t[:, 0].tolist() == want
    # every draft rejected: the residual of two rows
    lower = target * torch.rand(target.shape, generator=g)
    lower[2] = 0.0
    two = torch.cat([target, target], 1)
    drafted = torch.full((R, 1), V // 3, dtype=torch.int32)
    uu = torch.cat([torch.full((R, 1), 3e38), u], 1)
    lower[:, 0, V // 3] = 1.0
    want = [_draw(_whole((target[r, 0] - lower[r, 0]).numpy()), u[r, 0]) for r in range(R)]
    a, t = _run(two, lower, drafted, uu)
    assert (a == 0).all() and t[:, 0].tolist() == want and (t[:, 1] == -1).all()


@pytest.mark.parametrize("V", [24576, 100003, 200003])
def test_every_end_of_a_piece_of_a_large_row(V):
    """Equal weights, the threshold at and around the ends of the row's 64 pieces and of their eighths."""
    piece = -(-V // 64)
    ends = {e for k in range(65) for e in (k * piece, k * piece + (k % 8) * -(-piece // 8))}
    at = sorted(v for e in ends for v in (e - 1, e, e + 1) if 0 <= v < V)
    # weights of 2^20 units: the threshold u V 2^20 for u = (v + 1/2) / V lies inside token v, whatever u's rounding (V 2^-24 < 1/2)
    u = torch.tensor([(v + 0.5) / V for v in at], dtype=torch.float64).float()[:, None]
    target = torch.full((1, 1, V), 2.0 ** -20).expand(len(at), 1, V)
    _, t = _run(target.to(DEV).contiguous(), None, torch.zeros((len(at), 0), dtype=torch.int32), u)
    assert t[:, 0].tolist() == at
