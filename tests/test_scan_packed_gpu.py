"""GPU parity of glinattn_selective_scan_packed with the fp64 oracle."""
import numpy as np
import pytest
import torch

from gated_deltanet_02_gb300 import glinattn_selective_scan, glinattn_selective_scan_packed
from gated_deltanet_02_gb300.glinattn import DEV_BAD_COUNT, DEV_BAD_SLOT
from oracle import layer_parts as L

from helpers import f64
from layer_parts_helpers import EPS32, HALF, close

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
MARK = 7.0


def case(lengths, D, N, act, seed=0, strided=False, pad=0, first=0, slow=False):
    g = torch.Generator().manual_seed(seed)
    n, R = first + sum(lengths) + pad, len(lengths)
    P = R + 3
    start = np.concatenate([[first], first + np.cumsum(lengths)]).astype(np.int32)
    randn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    rank = -(-D // 16)
    off = 0 if strided else None
    rows, proj = randn(n, 2 * D).to(act).to(DEV), randn(n, rank + 2 * N).to(act).to(DEV)
    x, z, B, C = rows[:, :D], rows[:, D:], proj[:, rank:rank + N], proj[:, rank + N:]
    if off is None:
        x, z, B, C = x.contiguous(), z.contiguous(), B.contiguous(), C.contiguous()
    step = torch.exp(torch.rand(D, generator=g) * 4.6 + np.log(1e-3 if slow else 5e-3))
    return dict(x=x, z=z, B=B, C=C, delta=randn(n, D).to(act).to(DEV), A=(-torch.arange(1, N + 1) * torch.exp(0.1 * randn(D, N))).to(DEV),
                bias=(step + torch.log(-torch.expm1(-step))).to(DEV), skip=randn(D).to(DEV), pool=randn(P, D, N).to(DEV),
                slots=torch.randperm(P, generator=g)[:R].to(torch.int32).to(DEV), q_start=torch.from_numpy(start).to(DEV), lengths=lengths)


def check(c, z=True, skip=True, bias=True, resume=None, count=None, update=True, outputs=True, status=0, q_start=True, max_len=None, out=None):
    act = c["x"].dtype
    pool = c["pool"].clone()
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = act if out is None else out
    y = torch.full(c["x"].shape, MARK, dtype=out, device=DEV) if outputs else None
    ints = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    pick = lambda on, name: c[name] if on else None  # noqa: E731
    top = max(c["lengths"]) if max_len is None else max_len
    got = glinattn_selective_scan_packed(c["x"], c["delta"], c["B"], c["C"], c["A"], pool, c["slots"], c["q_start"] if q_start else None,
                                         max_q_len=top, z=pick(z, "z"), skip=pick(skip, "skip"), delta_bias=pick(bias, "bias"),
                                         resume=ints(resume), count=ints(count), update_state=update, outputs=outputs, y=y, dev_status=word)
    assert got is y and int(word.item()) == status
    want, ysize, new, psize, decay = L.scan_packed(f64(c["x"]), f64(c["delta"]), f64(c["B"]), f64(c["C"]), f64(c["A"]), f64(c["pool"]),
                                                   c["slots"].cpu().numpy(), c["q_start"].cpu().numpy(), f64(pick(z, "z")),
                                                   f64(pick(skip, "skip")), f64(pick(bias, "bias")), resume, count, top)
    # A decay is off by 2^-22 of itself at most (its argument, below 1 in magnitude where that matters, and the exponential),
    # a term dt B x by 2^-21 (softplus 2^-22, three roundings).  A state holds the products of at most min(rows, 1 / (1 - decay))
    # decays that matter, each step with a rounding more; y adds N products, skip and gate.
    steps = min(max(c["lengths"] + [1]), 1.0 / max(1e-9, 1.0 - decay))
    rel = (5.0 * steps + 8.0) * EPS32 * 2
    ref_pool = new if update else f64(c["pool"])
    touched = ref_pool != f64(c["pool"])
    close(pool, ref_pool, np.where(touched, rel * psize, 0.0), "pool")
    if outputs:
        N = c["A"].shape[1]
        tol = (rel + (N + 16) * EPS32) * ysize + HALF[out] * np.abs(want) + 1e-37
        run = ~np.isnan(want)
        close(y, np.where(run, want, MARK), np.where(run, tol, 0.0), "y")
    return y, pool


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("D", [1, 24, 130, 512])
@pytest.mark.parametrize("lengths", [[1], [1, 2, 0, 3, 1, 0], [63, 1, 64, 65, 128, 0, 31], [300, 5]], ids=["one", "short", "ends", "long"])
def test_packed(lengths, D, N, act):
    c = case(lengths, D, N, act, seed=D + N)
    check(c, resume=[int(r % 3 != 1) for r in range(len(lengths))])
    check(c, z=False, skip=False, bias=False, out=torch.float32)


def test_a_long_prompt():
    """Slow channels too: steps of 0.001."""
    check(case([3001], 48, 16, torch.float32, seed=1, slow=True), resume=[0])


@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
def test_long_and_short_requests(act, N):
    """Requests that are run in pieces beside short ones, ends at and around a piece's; some continue, some run in part."""
    lengths = [1500, 3, 0, 2049, 512, 513, 1024, 1025, 1, 1100]
    c = case(lengths, 40, N, act, seed=N, strided=True, pad=3, first=2)
    check(c, resume=[r % 3 != 1 for r in range(10)])
    check(c, count=[1500, 2, 0, 1537, 512, 0, 1000, 1025, 1, 512])
    c["slots"][3] = -1
    c["q_start"][-1] = 1 << 20
    check(c, status=DEV_BAD_SLOT | DEV_BAD_COUNT, max_len=2100)


def test_two_calls_with_one_workspace_on_one_stream():
    """A workspace's leftovers reach no later call; a larger one than needed serves too."""
    ws = torch.full((1 << 24,), 0xff, dtype=torch.uint8, device=DEV)
    for seed, n in ((21, 2500), (22, 1200)):
        c = case([n, 40], 64, 16, torch.bfloat16, seed=seed)
        args = c["x"], c["delta"], c["B"], c["C"], c["A"]
        p1, p2 = c["pool"].clone(), c["pool"].clone()
        a = glinattn_selective_scan_packed(*args, p1, c["slots"], c["q_start"], max_q_len=n, workspace=ws)
        b = glinattn_selective_scan_packed(*args, p2, c["slots"], c["q_start"], max_q_len=n)
        assert torch.equal(a, b) and torch.equal(p1, p2) and bool(torch.isfinite(a.float()).all())


def test_many_requests():
    lengths = [r % 4 for r in range(700)]
    check(case(lengths, 40, 16, torch.bfloat16, seed=2))
    check(case([1] * 333, 264, 16, torch.bfloat16, seed=3))


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 100, 33])
def test_slices(D, act):
    check(case([70, 1, 0, 9], D, 16, act, seed=D, strided=True))


@pytest.mark.parametrize("R", [1, 5, 300])
@pytest.mark.parametrize("D", [256, 77])
def test_single_tokens_without_ranges(R, D):
    c = case([1] * R, D, 16, torch.bfloat16, seed=R)
    a, b = check(c, q_start=False), check(c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_padding_and_rows_before_the_first_request():
    check(case([3, 0, 68], 72, 16, torch.bfloat16, seed=4, pad=5, first=3))


@pytest.mark.parametrize("N", [8, 16, 32])
def test_verified_and_replayed_drafts(N):
    lengths = [5, 5, 1, 5, 3, 5]
    c = case(lengths, 136, N, torch.bfloat16, seed=N)
    accept = [0, 5, 1, 2, 3, 1]
    whole, _ = check(c, update=False)
    _, pool = check(c, count=accept, outputs=False)
    part, pool2 = check(c, count=accept)
    assert torch.equal(pool, pool2)
    at = 0
    for n, a in zip(lengths, accept):
        assert torch.equal(part[at:at + a], whole[at:at + a]) and bool((part[at + a:at + n] == MARK).all())
        at += n


def test_replayed_drafts_equal_single_steps():
    """The state of a accepted drafts is that of a calls with one token each, bit for bit."""
    lengths, accept = [4, 4, 4], [1, 4, 2]
    c = case(lengths, 200, 16, torch.bfloat16, seed=11)
    _, pool = check(c, count=accept, outputs=False)
    step = c["pool"].clone()
    for k in range(4):
        on = [r for r in range(3) if accept[r] > k]
        if not on:
            break
        rows = torch.tensor([4 * r + k for r in on], device=DEV)
        pick = lambda name: c[name][rows].contiguous()  # noqa: E731
        glinattn_selective_scan_packed(pick("x"), pick("delta"), pick("B"), pick("C"), c["A"], step, c["slots"][on].contiguous(),
                                       delta_bias=c["bias"])
    assert torch.equal(pool, step)


@pytest.mark.parametrize("D", [40, 1024])
def test_pieces_equal_the_whole(D):
    """A prompt in pieces against the whole: the same recurrence, other places where pieces are joined."""
    c = case([200], D, 16, torch.float32, seed=12)
    y, pool = check(c)
    p2, at, out = c["pool"].clone(), 0, []
    for n in (1, 7, 64, 100, 28):
        s = slice(at, at + n)
        out.append(glinattn_selective_scan_packed(c["x"][s], c["delta"][s], c["B"][s], c["C"][s], c["A"], p2, c["slots"],
                                                  torch.tensor([0, n], dtype=torch.int32, device=DEV), max_q_len=n, z=c["z"][s],
                                                  skip=c["skip"], delta_bias=c["bias"]))
        at += n
    *_, psize, _ = L.scan_packed(f64(c["x"]), f64(c["delta"]), f64(c["B"]), f64(c["C"]), f64(c["A"]), f64(c["pool"]),
                                 c["slots"].cpu().numpy(), c["q_start"].cpu().numpy(), bias=f64(c["bias"]))
    assert (np.abs(f64(p2) - f64(pool)) <= 2e-4 * psize + 1e-37).all()
    assert float((torch.cat(out) - y).abs().max()) <= 1e-4 * float(y.abs().max())


def test_equal_to_the_plain_scan():
    """Without bias, skip and gate it is glinattn_selective_scan on a batch of equal lengths."""
    B, T, D, N = 3, 130, 96, 16
    c = case([T] * B, D, N, torch.float32, seed=13)
    y, h = glinattn_selective_scan(c["x"].view(B, T, D), c["delta"].view(B, T, D), c["B"].view(B, T, N), c["C"].view(B, T, N), c["A"],
                                   c["pool"][c["slots"].long()])
    pool = c["pool"].clone()
    y2 = glinattn_selective_scan_packed(c["x"], c["delta"], c["B"], c["C"], c["A"], pool, c["slots"], c["q_start"])
    assert float((y2 - y.view(-1, D)).abs().max()) <= 2e-5 * float(y.abs().max())
    assert float((pool[c["slots"].long()] - h).abs().max()) <= 2e-5 * float(h.abs().max())


def test_no_pool():
    c = case([70, 0, 20], 48, 16, torch.float32, seed=14)
    y = glinattn_selective_scan_packed(c["x"], c["delta"], c["B"], c["C"], c["A"], q_start=c["q_start"], z=c["z"])
    p = c["pool"].clone()
    y2 = glinattn_selective_scan_packed(c["x"], c["delta"], c["B"], c["C"], c["A"], p, c["slots"], c["q_start"], z=c["z"],
                                        resume=torch.zeros(3, dtype=torch.int32, device=DEV), update_state=False)
    assert torch.equal(y, y2) and torch.equal(p, c["pool"])


def test_bad_requests_are_flagged_and_skipped():
    c = case([3, 70, 4, 2, 5], 64, 16, torch.float32, seed=5)
    c["slots"][1] = c["pool"].shape[0]
    c["slots"][3] = -1
    check(c, status=DEV_BAD_SLOT)
    c = case([3, 70, 4, 2, 5], 64, 16, torch.float32, seed=6)
    check(c, count=[3, 71, 4, -1, 2], status=DEV_BAD_COUNT)
    check(c, max_len=5, status=DEV_BAD_COUNT)                 # the second request is longer than it may be
    check(c, max_len=0, status=DEV_BAD_COUNT)
    c["q_start"][-1] = 1000
    check(c, status=DEV_BAD_COUNT, max_len=2000)


def test_decreasing_ranges_stay_in_bounds():
    """Valid ranges that overlap, between invalid ones: more pieces than there are rows for; flagged, nothing outside is touched."""
    n, R = 2000, 17
    c = case([n] + [0] * (R - 1), 40, 16, torch.bfloat16, seed=16)
    c["q_start"].copy_(torch.tensor([0, n] * 9, dtype=torch.int32)[:R + 1])
    for max_len, q_start in ((n, c["q_start"]), (4, c["q_start"] // 500)):
        word, pool = torch.zeros(1, dtype=torch.int32, device=DEV), c["pool"].clone()
        glinattn_selective_scan_packed(c["x"], c["delta"], c["B"], c["C"], c["A"], pool, c["slots"], q_start.to(torch.int32), max_q_len=max_len,
                                       dev_status=word)
        torch.cuda.synchronize()
        assert int(word.item()) == DEV_BAD_COUNT
        other = torch.ones(len(pool), dtype=torch.bool, device=DEV)
        other[c["slots"].long()] = False
        assert torch.equal(pool[other], c["pool"][other])


@pytest.mark.parametrize("act,N", [(torch.bfloat16, 16), (torch.float32, 32), (torch.float32, 8)])
@pytest.mark.parametrize("R,top", [(3, 11), (3, 12), (200, 24), (200, 25)])
def test_ends_of_the_kernels_ranges(R, top, act, N):
    """The longest requests that the kernel for few rows takes, and the shortest that the other does."""
    check(case([(7 * r) % (top + 1) for r in range(R - 1)] + [top], 72, N, act, seed=top), resume=[int(r % 3 != 1) for r in range(R)])


def test_special_values():
    """Steps far to either side, an infinity and NaN stay in their channel and behind their row."""
    c = case([40], 24, 16, torch.float32, seed=15)
    c["delta"][:, 2] = -200.0                                   # no step: the state stays
    c["delta"][:, 3] = 80.0                                     # a step after which nothing is left of the state
    c["x"][10, 5] = float("nan")
    c["x"][11, 6] = float("inf")
    pool = c["pool"].clone()
    y = glinattn_selective_scan_packed(c["x"], c["delta"], c["B"], c["C"], c["A"], pool, c["slots"], c["q_start"])
    with np.errstate(invalid="ignore"):
        want, ysize, new, psize, _ = L.scan_packed(f64(c["x"]), f64(c["delta"]), f64(c["B"]), f64(c["C"]), f64(c["A"]), f64(c["pool"]),
                                                   c["slots"].cpu().numpy(), c["q_start"].cpu().numpy())
    s = int(c["slots"][0])
    assert torch.equal(pool[s, 2], c["pool"][s, 2])
    assert np.isnan(f64(pool)[s, 5]).all() and np.isfinite(f64(y)[:10, 5]).all() and np.isnan(f64(y)[10:, 5]).all()
    assert not np.isfinite(f64(pool)[s, 6]).any() or not np.isfinite(new[s, 6]).all()
    fine = np.array([k not in (5, 6) for k in range(24)])
    assert (np.abs(f64(y) - want)[:, fine] <= 1e-4 * ysize[:, fine] + 1e-37).all()
    assert (np.abs(f64(pool)[s] - new[s])[fine] <= 1e-4 * psize[s][fine] + 1e-37).all()


def test_far_rows_pass_32_bit_offsets():
    D, N = 8192, 8
    n = (1 << 31) // D + 3
    x = torch.zeros((n, D), dtype=torch.bfloat16, device=DEV)
    x[-2:] = torch.randn((2, D), device=DEV).to(torch.bfloat16)
    B, C = torch.ones((n, N), dtype=torch.bfloat16, device=DEV), torch.ones((n, N), dtype=torch.bfloat16, device=DEV)
    A = -torch.ones((D, N), device=DEV)
    qs = torch.tensor([0, n - 2, n], dtype=torch.int32, device=DEV)
    y = glinattn_selective_scan_packed(x, x, B, C, A, q_start=qs, max_q_len=n, skip=torch.ones(D, device=DEV))
    xs = f64(x[-2:])
    want, ysize, *_ = L.scan_packed(xs, xs, np.ones((2, N)), np.ones((2, N)), f64(A), None, None, np.array([0, 2]), skip=np.ones(D))
    close(y[-2:], want, HALF[torch.bfloat16] * np.abs(want) + 64 * EPS32 * ysize)
    assert not bool(y[:-2].any())
