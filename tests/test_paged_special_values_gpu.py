"""Paged attention where scores, scales, pages or queries are out of the ordinary."""
import math

import numpy as np
import pytest
import torch

from gated_deltanet_02_gb300 import glinattn_paged_attention
from gated_deltanet_02_gb300.glinattn import DEV_BAD_SLOT
from oracle import paged as P

from paged_helpers import HALF_BF16, attention_tolerance, cache_args, dev, paged_case, rows_of

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _q(c, H, seed=1, size=2.0):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn((c["num_tok"], H, c["d"]), generator=g)).to(torch.bfloat16)


def _run(c, q, **kw):
    g = dev(c)
    args, scales = cache_args(g)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw.setdefault("max_q_len", max([n for n, _ in c["lengths"]], default=0))
    o = torch.full_like(q, 7.0).to(DEV)
    glinattn_paged_attention(q.to(DEV), *args, **scales, dev_status=status, o=o, **kw)
    torch.cuda.synchronize()
    return o.cpu(), int(status.item())


def _oracle(c, q, scale=None):
    sc = 1.0 / math.sqrt(c["d"]) if scale is None else scale
    qd = q.double().numpy()
    want, a = P.attention(qd, rows_of(c, "k"), rows_of(c, "v"), c["q_start"], c["kv_len"], sc)
    return want, attention_tolerance(c, qd, want, a, sc)


def _check(c, q, scale=None, extra=0.0, **kw):
    got, status = _run(c, q, scale=scale, **kw)
    assert status == 0
    want, tol = _oracle(c, q, scale)
    err = np.abs(got.double().numpy() - want)
    assert (err <= tol + extra).all(), (np.nanmax(err / (tol + extra)), int(np.isnan(err).sum()))
    return got


def _set(c, name, r, pos, x):
    """The row of request r at a position as x (every head), bf16 or e4m3 with scale 1."""
    at = (int(c["table"][r, pos // c["page"]]), slice(None), pos % c["page"])
    t = c[name + "_cache"]
    if c["cache"] == "e4m3":
        t.view(torch.uint8)[at] = torch.as_tensor(x).expand(c["Hkv"], c["d"]).to(torch.float8_e4m3fn).view(torch.uint8)
        c[name + "_scale"][at] = 127
    else:
        t[at] = torch.as_tensor(x, dtype=t.dtype).expand(c["Hkv"], c["d"])


#: one request, its items cut into single tiles; many requests, most items whole
FEW_AND_MANY = [1, 150]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [2, 140])
@pytest.mark.parametrize("R", FEW_AND_MANY)
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_query_with_nan_gives_nan(value, R, n, cache):
    """However its item is shared out; no other row is touched."""
    c = paged_case([(n, n + 300)] * R, 1, 128, 16, cache, seed=1)
    q = _q(c, 2)
    want, _ = _run(c, q)
    assert not bool(want.isnan().any())
    rows = [0, n - 1, c["num_tok"] - 1]
    q[rows, 1, 5] = value
    got, status = _run(c, q)
    assert status == 0
    clear = torch.ones(got.shape[:2], dtype=torch.bool)
    clear[rows, 1] = False
    # an infinite element of q gives scores of both infinities, so NaN
    assert bool(got[rows, 1].isnan().all())
    assert torch.equal(got[clear], want[clear])


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [2, 140])
@pytest.mark.parametrize("R", FEW_AND_MANY)
@pytest.mark.parametrize("tile", [0, 1, 3])
def test_keys_that_are_all_nan_in_a_tile(tile, R, n, cache):
    """Every row that sees the tile is NaN, whether or not the tile is a piece of its own."""
    c = paged_case([(n, 520 + n)] * R, 1, 64, 16, cache, seed=2)
    r = R // 2
    for t in range(128 * tile, 128 * tile + 128):
        at = (int(c["table"][r, t // 16]), 0, t % 16)
        if cache == "e4m3":
            c["k_scale"][at] = 255
        else:
            c["k_cache"][at] = math.nan
    q = _q(c, 4)
    got, status = _run(c, q)
    assert status == 0
    mine = torch.zeros(c["num_tok"], dtype=torch.bool)
    mine[n * r:n * (r + 1)] = True
    assert bool(got[mine].isnan().all()) and not bool(got[~mine].isnan().any())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("R", FEW_AND_MANY)
def test_a_bad_page_that_only_later_rows_read(R, d, cache):
    """256 rows an item: the last 128 read the page and stay as they were, the first 128 do not read it."""
    c = paged_case([(256, 256)] * R, 1, d, 16, cache, seed=3)
    q = _q(c, 1)
    want, status = _run(c, q)
    assert status == 0
    r = R // 2
    c["table"][r, 11] = c["pages"]
    for _ in range(5):
        got, status = _run(c, q)
        assert status == DEV_BAD_SLOT
        lost = torch.zeros(c["num_tok"], dtype=torch.bool)
        lost[256 * r + 128:256 * (r + 1)] = True
        assert bool((got[lost] == 7).all())
        assert torch.equal(got[~lost], want[~lost])


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 3, 140])
@pytest.mark.parametrize("kv", [0, 90, 700])
@pytest.mark.parametrize("level", [-60.0, -90.0, -400.0, 400.0])
def test_scores_far_from_zero(level, kv, n, cache):
    """Softmax does not depend on a common term of the scores."""
    c = paged_case([(n, kv + n), (n, n)], 2, 128, 16, cache, seed=4, fill=0.5)
    u = level / (4.0 * math.sqrt(128))               # 4 u sqrt(128): the common term
    for name in ("k",):
        rows = [torch.from_numpy(x) for x in rows_of(c, name)]
        for r, x in enumerate(rows):
            for t in range(len(x)):
                at = (int(c["table"][r, t // 16]), slice(None), t % 16)
                if cache == "e4m3":
                    v, e = P.quantise((x[t] + u).numpy())
                    c["k_cache"].view(torch.uint8)[at] = torch.from_numpy(v).float().to(torch.float8_e4m3fn).view(torch.uint8)
                    c["k_scale"][at] = torch.from_numpy(e + 127).to(torch.uint8)
                else:
                    c["k_cache"][at] = (x[t] + u).to(torch.bfloat16)
    q = (4.0 + 0.25 * torch.randn((c["num_tok"], 8, 128), generator=torch.Generator().manual_seed(5))).to(torch.bfloat16)
    _check(c, q)


def _repeat(c, R):
    """The case's requests R times over, all over the same pages."""
    n = c["num_tok"]
    start = torch.cat([c["q_start"][:-1] + n * i for i in range(R)] + [torch.tensor([n * R], dtype=torch.int32)])
    return dict(c, lengths=c["lengths"] * R, num_tok=n * R, table=c["table"].repeat(R, 1), kv_len=c["kv_len"].repeat(R), q_start=start)


def _check_repeated(c, q, R, extra=0.0):
    """Against the oracle with the requests once, and R times over (items cut differently, many tiles each)."""
    want, tol = _oracle(c, q)
    got, status = _run(_repeat(c, R), q.repeat(R, 1, 1))
    assert status == 0
    err = np.abs(got.double().numpy().reshape(R, *q.shape) - want) / (tol + extra)
    assert (err <= 1).all(), (np.nanmax(err), int(np.isnan(err).sum()))


@pytest.mark.parametrize("R", [1, 150])
@pytest.mark.parametrize("n", [1, 5, 140])
@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("codes", [(160, 27), (246, 27), (246, 127), (246, 110), (127, 27), (150, 20 + 27)])
def test_value_scales_far_apart(codes, order, n, R):
    """Few value rows of a large scale among many of a small one, or of zeros: no key is missing from the sum."""
    c = paged_case([(n, 700 + n)] + [(n, 60 + n)] * 3, 1, 64, 16, "e4m3", seed=6)
    g = torch.Generator().manual_seed(7)
    c["v_scale"][:] = codes[1]
    if codes[1] == 27:
        c["v_cache"].view(torch.uint8)[:] = 0        # rows of zeros have the smallest scale
    for r, (_, kv) in enumerate(c["lengths"]):
        at = [3, 40, 190, 640] if order == 1 else [kv - n - 1]
        for t in at:
            if t < kv:
                cell = (int(c["table"][r, t // 16]), 0, t % 16)
                c["v_scale"][cell] = codes[0]
                x = torch.randn(64, generator=g) * 100
                c["v_cache"].view(torch.uint8)[cell] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    _check_repeated(c, _q(c, 2, size=1.0), R)


@pytest.mark.parametrize("n,H", [(1, 8), (3, 8), (5, 8), (40, 8)])
@pytest.mark.parametrize("bits", [8, 14, 16, 18, 20, 22, 26])
@pytest.mark.parametrize("R", [1, 320])
def test_one_key_over_a_flat_tail(R, bits, n, H):
    """A key far above some 32,000 equal ones, whose weights add up, over an e4m3 cache: one request, cut into
    single tiles, and many over the same pages, each in one or two pieces."""
    kv = 32768
    c = paged_case([(n, kv)], 1, 64, 64, "e4m3", seed=8)
    g = torch.Generator().manual_seed(9)
    c["k_cache"].view(torch.uint8)[:] = 0
    _set(c, "k", 0, 77, bits * math.log(2.0) * 8.0 / 64.0)       # q of ones, scale 1 / 8
    c["v_scale"][:] = 127
    c["v_cache"] = (1.0 + 0.2 * torch.rand(c["v_cache"].shape, generator=g)).to(torch.float8_e4m3fn)
    _set(c, "v", 0, 77, -1.0)
    q = torch.ones((n, H, 64), dtype=torch.bfloat16)
    _check_repeated(c, q, R)


@pytest.mark.parametrize("n,H", [(1, 8), (5, 8), (40, 8)])
@pytest.mark.parametrize("R", [1, 200])
@pytest.mark.parametrize("spread", [0, 4, 8, 12, 16, 20])
def test_sparse_value_rows_of_other_scales(spread, n, H, R):
    """A row of a large scale that is zero in half of the channels: the others' values there are not lost."""
    c = paged_case([(n, 300 + n)], 1, 64, 16, "e4m3", seed=10)
    c["v_scale"][:] = 127
    big = torch.zeros(64)
    big[:32] = 300.0
    for t in (5, 150, 290):
        _set(c, "v", 0, t, big)
        c["v_scale"][int(c["table"][0, t // 16]), 0, t % 16] = 127 + spread
    q = _q(c, H, size=0.5)
    # a weight times its value's scale is held to 2^-33 of the row's largest such product, once a key
    floor = 2.0 ** -33 * (300 + n) * 448.0 * 2.0 ** spread
    _check_repeated(c, q, R, extra=floor)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [2, 140])
@pytest.mark.parametrize("scale", [1e-12, 1e-20, 1e-30, 1e-38])
def test_tiny_scales_and_rows_of_zeros(scale, n, cache):
    """Queries of zeros, or scores of next to nothing: the mean of the visible values."""
    c = paged_case([(n, 200), (n, n)], 1, 128, 16, cache, seed=11)
    q = _q(c, 4)
    q[::3] = 0.0
    _check(c, q, scale=scale)


def _set_all(c, name, x):
    """Every row of the pool as x [d], quantised for an e4m3 cache."""
    if c["cache"] == "e4m3":
        v, e = P.quantise(np.asarray(x, np.float64)[None])
        c[name + "_cache"].view(torch.uint8)[:] = torch.from_numpy(v[0]).float().to(torch.float8_e4m3fn).view(torch.uint8)
        c[name + "_scale"][:] = int(e[0]) + 127
    else:
        c[name + "_cache"][:] = torch.as_tensor(x, dtype=torch.float64).to(torch.bfloat16)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 3, 140])
@pytest.mark.parametrize("R", [1, 100])
@pytest.mark.parametrize("size", [-1e30, 1e30, -3.3e8, 7.7e10, 1e4])
def test_equal_scores_of_any_size_share_the_weight(size, R, n, cache):
    """Keys that are all masked by a huge negative value, or all huge: the mean of the visible values, over many
    tiles and pieces."""
    c = paged_case([(n, 600 + n), (n, 90 + n)], 1, 128, 16, cache, seed=12)
    _set_all(c, "k", np.full(128, size))
    H = 4
    q = (torch.tensor([0.37, 0.53, 1.0, 0.01])[None, :, None] * torch.ones((c["num_tok"], H, 128))).to(torch.bfloat16)
    # equal keys have equal scores, whatever their rounding: sums of 128 equal products are exact up to a common factor
    v = rows_of(c, "v")
    want = np.concatenate([np.stack([v[r][:kv - n + i + 1, 0].mean(0) for i in range(n)]) for r, (_, kv) in enumerate(c["lengths"])])
    size_a = np.concatenate([np.stack([np.abs(v[r][:kv - n + i + 1, 0]).mean(0) for i in range(n)]) for r, (_, kv) in enumerate(c["lengths"])])
    got, status = _run(_repeat(c, R), q.repeat(R, 1, 1))
    assert status == 0
    err = np.abs(got.double().numpy().reshape(R, *q.shape) - want[:, None])
    # the output's rounding, the weights', 2^-20 for the exponential and the sums
    tol = HALF_BF16 * np.abs(want) + (HALF_BF16 + 2.0 ** -20) * size_a + 1e-30
    assert (err <= tol[:, None]).all(), (np.nanmax(err / tol[:, None]), int(np.isnan(err).sum()))


@pytest.mark.parametrize("n", [1, 140])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_saturated_keys_in_an_e4m3_cache(sign, n):
    """A key row with an infinite element is stored as +-448 2^119: it takes all the weight, or none."""
    c = paged_case([(n, 300 + n)], 1, 64, 16, "e4m3", seed=13)
    x = torch.zeros(64)
    x[5] = 448.0 * sign
    _set(c, "k", 0, 33, x)
    c["k_scale"][int(c["table"][0, 2]), 0, 1] = 246
    q = _q(c, 2, size=0.5).abs()
    q[:, :, 5] = 1.5
    v = rows_of(c, "v")[0]
    if sign > 0:
        got, status = _run(c, q)
        assert status == 0
        want = np.broadcast_to(v[33, 0], (n, 2, 64))
        assert (np.abs(got.double().numpy() - want) <= 2.0 ** -7 * np.abs(want)).all()   # a weight's and the output's rounding
    else:
        got, status = _run(c, q)
        assert status == 0
        c["k_scale"][int(c["table"][0, 2]), 0, 1] = 127       # -448: no weight either
        want, tol = _oracle(c, q)
        assert (np.abs(got.double().numpy() - want) <= tol).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 3, 140])
@pytest.mark.parametrize("R", [1, 100])
@pytest.mark.parametrize("rise", [0.0, 3.0, 5.0])
def test_values_next_to_the_largest(rise, R, n, cache):
    """A value of 3e38 (an infinite one as an e4m3 cache stores it) does not overflow, also where its key's score
    is above all before it by less than what moves the running maximum (rise, in nats)."""
    c = paged_case([(n, 300 + n), (n, 200 + n)], 1, 128, 16, cache, seed=14)
    for name in ("k", "v"):
        _set_all(c, name, np.zeros(128))
    x = torch.zeros(128)
    for r in range(2):
        _set(c, "k", r, 180, math.sqrt(128) * rise / 128)          # q of ones
        if cache == "e4m3":
            x[3], x[70] = 448.0, -448.0
            _set(c, "v", r, 180, x)
            c["v_scale"][int(c["table"][r, 180 // 16]), 0, 180 % 16] = 246
        else:
            x[3], x[70] = 3e38, -3e38
            _set(c, "v", r, 180, x)
    q = torch.ones((c["num_tok"], 2, 128), dtype=torch.bfloat16)
    _check_repeated(c, q, R)


def _set_row(c, r, t, x):
    """The key row of request r at a position as x [d], quantised for an e4m3 cache."""
    if c["cache"] == "bf16":
        _set(c, "k", r, t, torch.from_numpy(x))
        return
    v, e = P.quantise(x[None])
    cell = (int(c["table"][r, t // c["page"]]), slice(None), t % c["page"])
    c["k_cache"].view(torch.uint8)[cell] = torch.from_numpy(v[0]).float().to(torch.float8_e4m3fn).view(torch.uint8)
    c["k_scale"][cell] = int(e[0]) + 127


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 3, 140])
@pytest.mark.parametrize("R", [1, 100])
@pytest.mark.parametrize("low", [-1e3, -1e6, -1e30])
def test_masked_keys_before_ordinary_ones(low, R, n, cache):
    """The first 200 keys are masked by a huge negative value: the ordinary ones after them keep their differences."""
    c = paged_case([(n, 500 + n), (n, 210 + n)], 1, 128, 16, cache, seed=15)
    q = _q(c, 4)
    q[:, :, 7] = 3.0

    def mask(value):
        x = np.zeros(128)
        x[7] = value
        for r in range(2):
            for t in range(200):
                _set_row(c, r, t, x)

    mask(-200.0)                             # no weight either, and a tolerance of ordinary scores
    want, tol = _oracle(c, q)
    mask(low)
    got, status = _run(_repeat(c, R), q.repeat(R, 1, 1))
    assert status == 0
    err = np.abs(got.double().numpy().reshape(R, *q.shape) - want) / tol
    assert (err <= 1).all(), (np.nanmax(err), int(np.isnan(err).sum()))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 3, 140])
@pytest.mark.parametrize("R", [1, 100])
@pytest.mark.parametrize("levels", [(1e30, 3e30, 7e30), (-7e30, -3e30, -1e30), (-1e30, 1e9, 7e9), (1e5, 1.1e7, 1.3e11)])
def test_levels_of_huge_scores(levels, R, n, cache):
    """Keys of three levels of scores far apart, each over several tiles: the mean of the values of the highest one seen."""
    c = paged_case([(n, 700 + n)], 1, 64, 16, cache, seed=16)
    kv = 700 + n
    level = np.where(np.arange(kv) < 150, 0, np.where(np.arange(kv) < 300, 1, 2))
    for t in range(kv):
        _set_row(c, 0, t, np.full(64, levels[level[t]]))
    q = (torch.tensor([0.37, 1.0])[None, :, None] * torch.ones((n, 2, 64))).to(torch.bfloat16)
    v = rows_of(c, "v")[0][:, 0]
    top = level == 2
    got, status = _run(_repeat(c, R), q.repeat(R, 1, 1))
    assert status == 0
    got = got.double().numpy().reshape(R, n, 2, 64)
    for i in range(n):
        rows = v[:kv - n + i + 1][top[:kv - n + i + 1]]
        tol = HALF_BF16 * np.abs(rows.mean(0)) + (HALF_BF16 + 2.0 ** -20) * np.abs(rows).mean(0)
        assert (np.abs(got[:, i] - rows.mean(0)) <= tol).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 3, 140])
@pytest.mark.parametrize("R", [1, 100])
def test_scores_that_overflow_to_minus_infinity(R, n, cache):
    """Scores are fp32: keys whose scores are below its range count as masked, and rows of them alone give zeros."""
    c = paged_case([(n, 400 + n)], 1, 64, 16, cache, seed=17)
    _set_all(c, "k", np.full(64, -1e33))
    q = torch.ones((n, 2, 64), dtype=torch.bfloat16)
    got, status = _run(_repeat(c, R), q.repeat(R, 1, 1), scale=1e5)
    assert status == 0 and bool((got == 0).all())
    _set_row(c, 0, 250, np.full(64, 1e-3))          # one ordinary key: all the weight
    got, status = _run(_repeat(c, R), q.repeat(R, 1, 1), scale=1e5)
    want = rows_of(c, "v")[0][250, 0]
    assert status == 0 and bool((np.abs(got.double().numpy() - want) <= 2.0 ** -7 * np.abs(want)).all())


@pytest.mark.parametrize("n", [1, 5, 140])
@pytest.mark.parametrize("R", [1, 100])
@pytest.mark.parametrize("size", [-1e30, -3e6, 4e7, 1e20])
@pytest.mark.parametrize("codes", [(100, 112), (125, 135), (140, 160), (60, 66), (190, 200)])
def test_value_scales_beside_huge_scores(codes, size, R, n):
    """Beside scores that leave no digits for a value's exponent: the mean of the visible values, as ever."""
    c = paged_case([(n, 600 + n)], 1, 64, 16, "e4m3", seed=18)
    _set_all(c, "k", np.full(64, size))
    g = torch.Generator().manual_seed(19)
    c["v_scale"] = torch.randint(codes[0], codes[1], c["v_scale"].shape, generator=g).to(torch.uint8)
    q = (torch.tensor([0.37, 1.0, 0.01])[None, :, None] * torch.ones((n, 3, 64))).to(torch.bfloat16)
    v = rows_of(c, "v")[0][:, 0]
    got, status = _run(_repeat(c, R), q.repeat(R, 1, 1))
    assert status == 0
    got = got.double().numpy().reshape(R, n, 3, 64)
    for i in range(n):
        rows = v[:600 + i + 1]
        tol = HALF_BF16 * np.abs(rows.mean(0)) + (HALF_BF16 + 2.0 ** -20) * np.abs(rows).mean(0)
        assert (np.abs(got[:, i] - rows.mean(0)) <= tol).all()
