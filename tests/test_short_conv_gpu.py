"""GPU parity of glinattn_short_conv with the fp64 oracle."""
import numpy as np
import pytest
import torch

from gated_deltanet_02_gb300 import glinattn_short_conv
from gated_deltanet_02_gb300.glinattn import DEV_BAD_COUNT, DEV_BAD_SLOT
from oracle import layer_parts as L

from helpers import f64
from layer_parts_helpers import EPS32, HALF, close

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
MARK = 7.0

LENGTHS = {
    "one": [1], "short": [1, 2, 3, 0, 4, 5, 1, 0, 0, 2], "ends": [15, 1, 16, 17, 14, 3, 31, 2, 33], "long": [333, 0, 1, 500],
    "many": [r % 4 for r in range(1100)],
}


def case(lengths, C, width, act, seed=0, stride=0, offset=0, pad=0, first=0):
    g = torch.Generator().manual_seed(seed)
    n, R = first + sum(lengths) + pad, len(lengths)
    P = R + 3
    start = np.concatenate([[first], first + np.cumsum(lengths)]).astype(np.int32)
    wide = torch.randn((n, max(stride, C + offset)), generator=g).to(act).to(DEV)
    return dict(x=wide[:, offset:offset + C], w=torch.randn((C, width), generator=g).to(DEV), bias=torch.randn(C, generator=g).to(DEV),
                pool=torch.randn((P, width - 1, C), generator=g).to(act).to(DEV),
                slots=torch.randperm(P, generator=g)[:R].to(torch.int32).to(DEV), q_start=torch.from_numpy(start).to(DEV), lengths=lengths)


def check(c, silu=True, bias=True, resume=None, count=None, update=True, outputs=True, status=0, q_start=True):
    x, w, act = c["x"], c["w"], c["x"].dtype
    pool = c["pool"].clone()
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = torch.full(x.shape, MARK, dtype=act, device=DEV) if outputs else None
    ints = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    got = glinattn_short_conv(x, w, c["bias"] if bias else None, pool, c["slots"], c["q_start"] if q_start else None, resume=ints(resume),
                              count=ints(count), silu=silu, update_state=update, outputs=outputs, y=y, dev_status=word)
    assert got is y and int(word.item()) == status
    want, size, new = L.short_conv(f64(x), f64(w), f64(c["bias"]) if bias else None, f64(c["pool"]), c["slots"].cpu().numpy(),
                                   c["q_start"].cpu().numpy(), resume, count, silu)
    close(pool, new if update else f64(c["pool"]), 0.0, "pool")      # copies of inputs: bit for bit
    if outputs:
        # a sum of width + 1 terms; SiLU's slope is at most 1.1, its own error (exponential, sum, quotient) 8 units
        tol = 1.1 * (w.shape[1] + 1) * EPS32 * size + (8 * EPS32 + HALF[act]) * np.abs(want) + 1e-37
        run = ~np.isnan(want)
        close(y, np.where(run, want, MARK), np.where(run, tol, 0.0), "y")
    return y, pool


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("C", [1, 40, 256, 301, 520])
@pytest.mark.parametrize("name", list(LENGTHS))
def test_packed(name, C, width, act):
    lengths = LENGTHS[name]
    if name == "many" and C not in (40, 301):
        pytest.skip("two channel counts for the large batch")
    c = case(lengths, C, width, act, seed=C + width)
    resume = [r % 3 != 1 for r in range(len(lengths))]
    check(c, resume=[int(v) for v in resume])
    check(c, silu=False, bias=False)


@pytest.mark.parametrize("C", [9000, 8999])
def test_many_channels_and_rows(C):
    """Enough work for tiles of many rows; requests that begin at every place of a tile."""
    check(case([15, 1, 16, 17, 14, 3, 31, 2, 33, 0, 700, 47], C, 4, torch.bfloat16, seed=C), resume=[0, 1] * 6)


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C,stride,offset", [(64, 136, 0), (64, 136, 72), (64, 137, 0), (64, 128, 3), (33, 70, 35)])
def test_slices(C, stride, offset, act):
    check(case([5, 40, 1, 0, 3], C, 4, act, seed=stride, stride=stride, offset=offset))


@pytest.mark.parametrize("R", [1, 5, 300])
@pytest.mark.parametrize("C", [2048, 77])
def test_single_tokens_without_ranges(R, C):
    c = case([1] * R, C, 4, torch.bfloat16, seed=R)
    a = check(c, q_start=False)
    b = check(c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_no_pool():
    c = case([4, 0, 20], 48, 4, torch.float32, seed=1)
    y = glinattn_short_conv(c["x"], c["w"], c["bias"], q_start=c["q_start"])
    want, size, _ = L.short_conv(f64(c["x"]), f64(c["w"]), f64(c["bias"]), None, None, c["q_start"].cpu().numpy())
    close(y, want, 1.1 * 5 * EPS32 * size + 9 * EPS32 * np.abs(want))


def test_padding_and_rows_before_the_first_request():
    check(case([3, 0, 18], 72, 4, torch.bfloat16, seed=4, pad=5, first=3))


@pytest.mark.parametrize("width", [2, 3, 4])
def test_verified_and_replayed_drafts(width):
    """Verifying leaves the pool; replaying the accepted drafts gives the state of as many steps."""
    lengths = [5, 5, 1, 5, 3, 5]
    c = case(lengths, 136, width, torch.bfloat16, seed=width)
    accept = [0, 5, 1, 2, 3, 1]
    whole, _ = check(c, update=False)
    _, pool = check(c, count=accept, outputs=False)
    part, pool2 = check(c, count=accept)
    assert torch.equal(pool, pool2)
    at = 0
    for n, a in zip(lengths, accept):
        assert torch.equal(part[at:at + a], whole[at:at + a]) and bool((part[at + a:at + n] == MARK).all())
        at += n


def test_pieces_equal_the_whole():
    c = case([37, 12], 264, 4, torch.bfloat16, seed=8)
    y, pool = check(c)
    p2, out = c["pool"].clone(), []
    x0, x1 = c["x"][:37], c["x"][37:]
    for cut in ((0, 1, 0, 2), (1, 3, 2, 2), (3, 20, 2, 11), (20, 37, 11, 12)):
        part = torch.cat([x0[cut[0]:cut[1]], x1[cut[2]:cut[3]]])
        qs = torch.tensor([0, cut[1] - cut[0], len(part)], dtype=torch.int32, device=DEV)
        out.append((cut, glinattn_short_conv(part, c["w"], c["bias"], p2, c["slots"], qs)))
    assert torch.equal(p2, pool)
    for cut, o in out:
        k = cut[1] - cut[0]
        assert torch.equal(o[:k], y[cut[0]:cut[1]]) and torch.equal(o[k:], y[37 + cut[2]:37 + cut[3]])


def test_bad_requests_are_flagged_and_skipped():
    c = case([3, 20, 4, 2, 5], 64, 4, torch.float32, seed=5)
    c["slots"][1] = c["pool"].shape[0]
    c["slots"][3] = -1
    check(c, status=DEV_BAD_SLOT)
    c = case([3, 20, 4, 2, 5], 64, 4, torch.float32, seed=6)
    check(c, count=[3, 21, 4, -1, 2], status=DEV_BAD_COUNT)
    c["q_start"][-1] = 1000                                   # the last request ends outside the rows
    check(c, status=DEV_BAD_COUNT)


def test_decreasing_ranges_stay_in_bounds():
    c = case([3, 20, 4, 2, 5], 64, 4, torch.float32, seed=7)
    c["q_start"][2] = 1
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    glinattn_short_conv(c["x"], c["w"], None, c["pool"], c["slots"], c["q_start"], dev_status=word)
    assert int(word.item()) == DEV_BAD_COUNT


def test_special_values_stay_in_their_channel():
    c = case([6, 6], 16, 4, torch.float32, seed=9)
    c["x"][2, 3] = float("nan")
    c["x"][8, 5] = float("inf")
    c["x"][9, 7] = -1e38
    x, w = f64(c["x"]), f64(c["w"])
    y = glinattn_short_conv(c["x"], c["w"], None, c["pool"].clone(), c["slots"], c["q_start"], silu=False)
    with np.errstate(invalid="ignore"):
        want, size, _ = L.short_conv(x, w, None, f64(c["pool"]), c["slots"].cpu().numpy(), c["q_start"].cpu().numpy(), act=False)
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(f64(y)), fine)
    assert (np.abs(f64(y) - want)[fine] <= (6 * EPS32 * size)[fine] + 1e-37).all()


def test_far_rows_pass_32_bit_offsets():
    C = 8192
    n = (1 << 31) // C + 5
    x = torch.zeros((n, C), dtype=torch.bfloat16, device=DEV)
    x[-6:] = torch.randn((6, C), device=DEV).to(torch.bfloat16)
    w = torch.randn((C, 4), device=DEV)
    qs = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    y = glinattn_short_conv(x, w, q_start=qs)
    want, size, _ = L.short_conv(f64(x[-9:]), f64(w), None, None, None, np.array([0, 9]))
    close(y[-6:], want[3:], (1.1 * 5 * EPS32 * size + (HALF[torch.bfloat16] + 8 * EPS32) * np.abs(want))[3:] + 1e-37)
    assert not bool(y[:-6].any())
