"""GPU parity of glinattn_accept_drafts with the oracle: whole numbers, equal."""
import numpy as np
import pytest
import torch

from gated_deltanet_02_gb300 import glinattn_accept_drafts
from gated_deltanet_02_gb300.glinattn import DEV_BAD_COUNT, DEV_BAD_PROB, DEV_BAD_TOKEN
from oracle import paged as P

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _case(R, D, V, seed, sharp=2.5):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((R, D + 1, V), generator=g) * sharp
    target = torch.softmax(z + 0.5 * torch.randn((R, D + 1, V), generator=g), -1)
    draft = torch.softmax(z[:, :D], -1)
    tokens = torch.multinomial(draft.reshape(R * D, V), 1, generator=g).reshape(R, D).to(torch.int32) if R * D else \
        torch.zeros((R, D), dtype=torch.int32)
    return target, draft, tokens, torch.rand((R, D + 1), generator=g)


def _run(target, draft, drafted, u, num=None, **kw):
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    a, t = glinattn_accept_drafts(to(target), to(draft), to(drafted), to(u), num_drafts=to(num), **kw)
    return a.cpu().numpy(), t.cpu().numpy()


def _check(target, draft, tokens, u, num=None):
    got = _run(target, draft, tokens, u, num)
    want = P.accept_drafts(target.numpy(), None if draft is None else draft.numpy(), tokens.numpy(), u.numpy(),
                           None if num is None else num.numpy())
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    return got


@pytest.mark.parametrize("V", [1, 2, 63, 64, 65, 1000, 4099])
@pytest.mark.parametrize("R,D", [(1, 0), (1, 1), (5, 4), (3, 40)])
def test_random_rounds(R, D, V):
    if D == 40 and V > 1000:
        pytest.skip("covered by the smaller vocabularies")
    target, draft, tokens, u = _case(R, D, V, 11 * R + D + V)
    num = torch.arange(R, dtype=torch.int32) * 3 % (D + 1)
    _check(target, draft, tokens, u)
    _check(target, draft, tokens, u, num)
    _check(target, None, tokens, u, num)


def test_many_requests_cover_every_accepted_length():
    target, draft, tokens, u = _case(300, 4, 257, 5)
    a, _ = _check(target, draft, tokens, u)
    assert set(a.tolist()) == {0, 1, 2, 3, 4}


def test_ends_of_the_uniform_range_and_rows_of_one_element():
    target, draft, tokens, u = _case(6, 3, 500, 8)
    u[0], u[1] = 0.0, 1.0 - 2.0 ** -24
    target[2] = 0.0
    target[2, :, 499] = 1.0                   # all mass on the last element
    target[3] = 0.0
    target[3, :, 0] = 1.0
    target[4, :, 100:] = 0.0                  # a tail without mass, the largest uniform
    u[4, 3] = 1.0 - 2.0 ** -24
    _check(target, draft, tokens, u)
    _check(target, None, tokens, u)


def test_equal_rows_leave_no_residual_and_fall_back_to_the_target():
    target, draft, tokens, u = _case(4, 2, 300, 9)
    draft[:] = target[:, :2]
    u[:, :2] = 1.0                            # u q < p fails where q = p: rejected with nothing left
    a, t = _check(target, draft, tokens, u)
    assert (a == 0).all()


def test_nan_and_values_past_one_count_as_documented():
    target, draft, tokens, u = _case(4, 2, 300, 10)
    target[0, :, 5] = float("nan")
    target[1, :, 7] = 3.0
    draft[2, :, 9] = float("nan")
    target[3, :, 11] = -1.0
    _check(target, draft, tokens, u)


def test_bad_counts_tokens_and_rows_are_flagged_and_skipped():
    target, draft, tokens, u = _case(5, 3, 200, 12)
    num = torch.tensor([3, 4, -1, 2, 3], dtype=torch.int32)
    tokens[3, 1] = 200                        # among the first two: bad
    tokens[4, 2] = 5
    tokens[0, 0] = 3
    target[4] = 0.0                           # no mass at all
    accept = torch.full((5,), 77, dtype=torch.int32, device=DEV)
    out = torch.full((5, 4), 88, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    a, t = _run(target, draft, tokens, u, num, accept=accept, tokens=out, dev_status=status)
    assert int(status.item()) == DEV_BAD_COUNT | DEV_BAD_TOKEN | DEV_BAD_PROB
    assert (a[1:] == 77).all() and (t[1:] == 88).all()
    want = P.accept_drafts(target[:1].numpy(), draft[:1].numpy(), tokens[:1].numpy(), u[:1].numpy())
    assert a[0] == want[0][0] and np.array_equal(t[0], want[1][0])


def test_a_token_behind_the_count_is_not_looked_at():
    target, draft, tokens, u = _case(3, 4, 100, 13)
    num = torch.tensor([2, 0, 4], dtype=torch.int32)
    tokens[0, 2:], tokens[1, :] = -5, 1000
    _check(target, draft, tokens, u, num)


def test_drawn_tokens_follow_the_target():
    """Acceptance and residual together draw from the target: over 20000 rounds
    a token's share is within 5 standard deviations of its probability."""
    V, R = 6, 20000
    g = torch.Generator().manual_seed(3)
    p = torch.softmax(torch.randn(V, generator=g), -1)
    q = torch.softmax(torch.randn(V, generator=g), -1)
    target = p.expand(R, 2, V).contiguous()
    draft = q.expand(R, 1, V).contiguous()
    tokens = torch.multinomial(q, R, replacement=True, generator=g).to(torch.int32).reshape(R, 1)
    _, t = _run(target, draft, tokens, torch.rand((R, 2), generator=g))
    share = np.bincount(t[:, 0], minlength=V) / R
    sd = np.sqrt(p.numpy() * (1 - p.numpy()) / R)
    assert (np.abs(share - p.numpy()) <= 5 * sd).all()


@pytest.mark.parametrize("scale", [2.0 ** -40, 2.0 ** -39, 2.0 ** -30, 2.0 ** -21, 2.0 ** -20, 2.0 ** -19, 1.0, 2.0 ** -126])
def test_whole_number_weights_at_every_size(scale):
    """Few units of 2^-40, weights around the border of their parts, subnormals, ones; every draw of a fine grid."""
    R, V = 400, 37
    g = torch.Generator().manual_seed(14)
    w = torch.rand((R, 1, V), generator=g) * 4 * scale
    w[:, :, 3] = scale
    w[:, :, 4] = scale * (1 - 2.0 ** -24)
    w[:, :, 5] = scale * (1 + 2.0 ** -23)
    w[:, :, 6] = 2.0 ** -149
    w[:, :, 7] = 2.0 ** -40
    w[:, :, 8] = 2.0 ** -41
    u = torch.arange(R, dtype=torch.float32)[:, None] / R
    _check(w, None, torch.zeros((R, 0), dtype=torch.int32), u)
    lower = w * torch.rand((R, 1, V), generator=g)   # a residual of two rows, every draft rejected
    two = torch.cat([w, w], 1)
    _check(two, lower, torch.full((R, 1), 6, dtype=torch.int32), torch.cat([torch.full((R, 1), 3e38), u], 1))
