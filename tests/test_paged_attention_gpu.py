"""GPU parity of glinattn_paged_attention with the fp64 oracle."""
import math

import numpy as np
import pytest
import torch

from gated_deltanet_02_gb300 import glinattn_paged_attention
from gated_deltanet_02_gb300 import glinattn as G
from gated_deltanet_02_gb300.glinattn import DEV_BAD_COUNT, DEV_BAD_SLOT
from oracle import paged as P

from paged_helpers import attention_tolerance, cache_args, dev, paged_case, rows_of

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
    o = glinattn_paged_attention(q.to(DEV), *args, **scales, dev_status=status, **kw)
    torch.cuda.synchronize()
    return o, int(status.item())


def _check(c, q, scale=None, **kw):
    sc = 1.0 / math.sqrt(c["d"]) if scale is None else scale
    o = torch.full_like(q, 7.0).to(DEV)
    got, status = _run(c, q, scale=scale, o=o, **kw)
    assert status == 0
    qd = q.double().numpy()
    want, a = P.attention(qd, rows_of(c, "k"), rows_of(c, "v"), c["q_start"], c["kv_len"], sc)
    got = got.double().cpu().numpy()
    out = np.isnan(want).all((1, 2))          # rows of no request
    assert (got[out] == 7.0).all()
    tol = attention_tolerance(c, qd, want, a, sc)
    bad = np.abs(got - want) > tol
    assert not bad[~out].any(), (np.abs(got - want)[~out] / tol[~out]).max()
    return got


MIXED = [(1, 40), (0, 7), (17, 17), (3, 130), (0, 0), (33, 295), (1, 128), (1, 129), (2, 1000)]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv,d,page", [(1, 1, 64, 16), (8, 2, 128, 16), (6, 2, 128, 32), (5, 5, 64, 64),
                                          (7, 1, 128, 128), (16, 1, 64, 16)])
def test_mixed_lengths(H, Hkv, d, page, cache):
    c = paged_case(MIXED, Hkv, d, page, cache, seed=2)
    _check(c, _q(c, H))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("kv", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 513, 3001])
def test_single_token(kv, cache):
    c = paged_case([(1, kv), (1, 1), (1, max(1, kv // 2))], 2, 128, 16, cache, seed=kv)
    _check(c, _q(c, 8))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len,kv,H,Hkv,d", [
    (64, 64, 4, 4, 128), (127, 127, 2, 2, 64), (128, 128, 2, 2, 128), (129, 129, 2, 1, 128), (257, 257, 3, 3, 64),
    (300, 700, 4, 1, 128), (256, 1111, 1, 1, 128), (65, 66, 8, 1, 64), (512, 512, 1, 1, 128), (90, 513, 6, 2, 128)])
def test_prompts_and_pieces(q_len, kv, H, Hkv, d, cache):
    c = paged_case([(q_len, kv), (1, 5), (q_len // 3, kv // 2 + 1)], Hkv, d, 16, cache, seed=q_len)
    _check(c, _q(c, H))


@pytest.mark.parametrize("q_len", [1, 2, 3, 4, 5, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_drafts_of_grouped_heads(q_len, cache):
    """Row counts q_len * H / Hkv around every tile size."""
    c = paged_case([(q_len, 400 + q_len), (q_len, q_len), (q_len, 131)], 1, 128, 32, cache, seed=q_len)
    _check(c, _q(c, 8))


@pytest.mark.parametrize("big", [False, True])
def test_rows_without_keys_give_zeros(big):
    n = 150 if big else 5
    c = paged_case([(n, 3), (2, 0), (n, 0), (n, 200)], 2, 64, 16, "bf16", seed=4)
    got = _check(c, _q(c, 4))
    assert (got[:n - 3] == 0).all() and (got[n:n + 2 + n] == 0).all()


@pytest.mark.parametrize("big", [False, True])
def test_padded_batch_and_rows_before_the_first_request(big):
    n = 140 if big else 3
    c = paged_case([(n, 160), (2, 9)], 2, 128, 16, "e4m3", seed=5, num_tok=n + 20, first=3)
    got = _check(c, _q(c, 4))
    assert (got[:3] == 7).all() and (got[n + 5:] == 7).all()


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_stale_rows_and_unread_pages_may_hold_nan(cache, big):
    """NaN and infinities behind kv_len, in the same page and in other pages."""
    q = 140 if big else 2
    c = paged_case([(q, 150), (1, 17), (q, 200)], 2, 128, 32, cache, seed=6)
    want = _check(c, _q(c, 4))
    live = torch.zeros((c["pages"], c["page"]), dtype=torch.bool)
    for r, (_, kv) in enumerate(c["lengths"]):
        for t in range(kv):
            live[int(c["table"][r, t // c["page"]]), t % c["page"]] = True
    for name in ("k", "v"):
        x = c[name + "_cache"].float()
        x.transpose(1, 2)[~live] = float("nan")
        c[name + "_cache"] = x.to(c[name + "_cache"].dtype)
        if cache == "e4m3":
            c[name + "_scale"].transpose(1, 2)[~live] = 255
    assert np.array_equal(_check(c, _q(c, 4)), want)


@pytest.mark.parametrize("big", [False, True])
def test_scores_of_minus_infinity(big):
    """Keys of -infinity score count as masked; a row of them alone gives zeros."""
    q = 130 if big else 2
    c = paged_case([(q, 300), (1, 40)], 1, 64, 16, "bf16", seed=7)
    for r, t in [(0, 0), (0, 5), (0, 129)] + [(1, t) for t in range(40)]:
        c["k_cache"][int(c["table"][r, t // 16]), 0, t % 16] = -float("inf")
    got = _check_inf(c, torch.ones((c["num_tok"], 2, 64), dtype=torch.bfloat16))
    assert (got[-1] == 0).all()


def _check_inf(c, q):
    got, status = _run(c, q)
    want, a = P.attention(q.double().numpy(), rows_of(c, "k"), rows_of(c, "v"), c["q_start"], c["kv_len"], 0.125)
    got = got.double().cpu().numpy()
    # |q| = 1: the scores' error is that of 64 products of |k| <= 5, 2^-24 each, doubled in the weights
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -9) * a).all()
    return got


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("size,scale", [(60.0, None), (2.0, 5.0), (1e-3, None), (2.0, 1e-4)])
def test_sharp_and_flat_scores(size, scale, big):
    """Scores of some hundreds (one key takes all the weight), and of nothing."""
    q = 140 if big else 3
    c = paged_case([(q, 500), (1, 300)], 2, 128, 16, "bf16", seed=8)
    _check(c, _q(c, 4, size=size), scale=scale)


@pytest.mark.parametrize("big", [False, True])
def test_growing_scores_rescale(big):
    """Keys whose scores grow along the cache: the running maximum moves in every tile."""
    q = 140 if big else 3
    c = paged_case([(q, 900)], 1, 128, 16, "bf16", seed=9)
    for t in range(900):
        c["k_cache"][int(c["table"][0, t // 16]), 0, t % 16] *= 1.0 + t / 60.0
    _check(c, _q(c, 4))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_scales_of_every_size(cache):
    """Values of very different magnitude from row to row."""
    c = paged_case([(2, 300), (140, 200)], 1, 128, 16, cache, seed=10)
    g = torch.Generator().manual_seed(3)
    if cache == "e4m3":
        c["v_scale"] = torch.randint(100, 150, c["v_scale"].shape, generator=g).to(torch.uint8)
    else:
        c["v_cache"] = c["v_cache"] * (2.0 ** torch.randint(-27, 23, c["v_cache"].shape[:3], generator=g))[..., None].to(torch.bfloat16)
    _check(c, _q(c, 4))
    _check(c, _q(c, 4), max_q_len=140)


@pytest.mark.parametrize("R,kv,H,Hkv", [(1, 40000, 8, 1), (2, 20011, 2, 2), (300, 37, 4, 2), (1, 700, 64, 8)])
def test_work_is_shared_out(R, kv, H, Hkv):
    """One long request over every SM; more requests than SMs."""
    c = paged_case([(1, kv - (r % 7)) for r in range(R)], Hkv, 64, 64, "bf16", seed=R)
    _check(c, _q(c, H))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len", [5, 15, 16, 17, 31])
def test_many_items_that_fill_half_a_row_tile(q_len, cache):
    """Several items per SM with 40 .. 248 of 256 rows, some with an empty second half."""
    c = paged_case([(max(1, q_len - 13 * (r % 2)), 60 + 5 * r) for r in range(160)], 2, 64, 16, cache, seed=q_len)
    q = _q(c, 16)
    first, status = _run(c, q)
    assert status == 0
    for _ in range(20):
        again, status = _run(c, q)
        assert status == 0 and torch.equal(again, first)
    c["lengths"] = c["lengths"][:6]
    n = int(c["q_start"][6])
    for k in ("kv_len", "table"):
        c[k] = c[k][:6].contiguous()
    c["q_start"], c["num_tok"] = c["q_start"][:7].contiguous(), n
    _check(c, q[:n].contiguous())


@pytest.mark.parametrize("big", [False, True])
def test_bad_pages_and_lengths_are_flagged_and_skipped(big):
    n = 150 if big else 2
    c = paged_case([(n, 200), (n, 200), (n, 200), (n, 200)], 2, 64, 16, "bf16", seed=11)
    q = _q(c, 4)
    good, _ = _run(c, q)
    c["table"][1, 0] = c["pages"]         # every query row reads it
    c["kv_len"][2] = 100000
    o = torch.full_like(q, 7.0).to(DEV)
    got, status = _run(c, q, o=o)
    assert status == DEV_BAD_SLOT | DEV_BAD_COUNT
    assert bool((got[n:3 * n] == 7).all())
    assert torch.equal(got[:n], good[:n]) and torch.equal(got[3 * n:], good[3 * n:])


def test_a_range_longer_than_max_q_len_is_flagged_and_skipped():
    c = paged_case([(2, 20), (5, 30), (1, 4)], 1, 128, 16, "bf16", seed=12)
    q = _q(c, 2)
    good, _ = _run(c, q)
    o = torch.full_like(q, 7.0).to(DEV)
    got, status = _run(c, q, o=o, max_q_len=4)
    assert status == DEV_BAD_COUNT
    assert bool((got[2:7] == 7).all()) and torch.equal(got[:2], good[:2]) and torch.equal(got[7:], good[7:])


def test_shared_pages():
    """Two requests over the same prefix pages."""
    c = paged_case([(2, 100), (3, 90)], 2, 128, 16, "e4m3", seed=13)
    c["table"][1, :4] = c["table"][0, :4]
    _check(c, _q(c, 4))


@pytest.mark.parametrize("big", [False, True])
def test_repeats_are_bit_identical_and_graphs_replay(big):
    n = 300 if big else 2
    c = paged_case([(n, 5000), (n, 3000), (1, 77)], 2, 128, 16, "bf16", seed=14)
    q = _q(c, 8)
    first, _ = _run(c, q)
    second, _ = _run(c, q)
    assert torch.equal(first, second)
    g = dev(c)
    args, _ = cache_args(g)
    a = G.PagedAttnArgs(G.BF16, 3, c["num_tok"], 8, 2, 128, 16, c["pages"], c["table"].shape[1], n, 0.1)
    need = G.library().glinattn_paged_attention_workspace_size(a)
    ws = torch.empty(max(1, need), dtype=torch.uint8, device=DEV)
    qd, o = q.to(DEV), torch.zeros_like(q).to(DEV)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        glinattn_paged_attention(qd, *args, max_q_len=n, o=o, workspace=ws)
        glinattn_paged_attention(qd, *args, max_q_len=n, o=o, workspace=ws)
    for _ in range(3):
        o.zero_()
        ws.fill_(255)                      # nothing is kept in the workspace between calls
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, first)
    # other lengths in the same buffers: the captured call reads them on the device
    g["kv_len"][0], g["kv_len"][2] = 4000, 50
    c["kv_len"][0], c["kv_len"][2] = 4000, 50
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, _run(c, q)[0])


def test_far_pages_pass_32_bit_offsets():
    """A pool of more than 2^32 bytes, the request in its last pages."""
    page, Hkv, d = 128, 8, 128
    pages = (1 << 32) // (page * Hkv * d * 2) + 3
    kc = torch.zeros((pages, Hkv, page, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    gen = torch.Generator(device=DEV).manual_seed(1)
    kc[-2:] = torch.randn((2, Hkv, page, d), generator=gen, device=DEV).to(torch.bfloat16)
    vc[-2:] = torch.randn((2, Hkv, page, d), generator=gen, device=DEV).to(torch.bfloat16)
    far = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device=DEV)
    near = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
    for n in (2, 100):
        kv, qs = torch.tensor([200], dtype=torch.int32, device=DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV)
        q = torch.randn((n, 8, d), generator=gen, device=DEV).to(torch.bfloat16)
        a = glinattn_paged_attention(q, kc, vc, far, kv, qs, max_q_len=n)
        b = glinattn_paged_attention(q, kc[-2:].clone(), vc[-2:].clone(), near, kv, qs, max_q_len=n)
        assert torch.equal(a, b) and float(a.abs().max()) > 0


@pytest.mark.parametrize("H,Hkv", [(130, 1), (256, 1), (96, 2)])
def test_large_groups(H, Hkv):
    """More heads per kv head than a row tile has rows."""
    c = paged_case([(3, 140), (1, 1), (2, 300)], Hkv, 64, 16, "bf16", seed=H)
    _check(c, _q(c, H))


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_outputs_at_a_16_byte_boundary(cache, big):
    n = 140 if big else 2
    c = paged_case([(n, 200), (n, 1000)], 2, 64, 32, cache, seed=15)
    q = _q(c, 4)
    want, _ = _run(c, q)
    flat = torch.full((q.numel() + 16,), 7.0, dtype=torch.bfloat16, device=DEV)
    o = flat[8:8 + q.numel()].view(q.shape)
    assert o.data_ptr() % 32 == 16
    _run(c, q, o=o)
    assert torch.equal(o, want) and bool((flat[:8] == 7).all()) and bool((flat[8 + q.numel():] == 7).all())


@pytest.mark.parametrize("big", [False, True])
def test_another_stream(big):
    """Outputs and workspace made by the call belong to the stream that it runs on."""
    n = 300 if big else 2
    c = paged_case([(n, 4000), (n, 900)], 2, 128, 16, "bf16", seed=16)
    q = _q(c, 8)
    want, _ = _run(c, q)
    g = dev(c)
    args, _ = cache_args(g)
    qd = q.to(DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        outs.append(glinattn_paged_attention(qd, *args, max_q_len=n, stream=side))
        torch.empty(64 << 20, dtype=torch.uint8, device=DEV).fill_(255)  # on the current stream
    side.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_two_calls_at_once():
    """Decode and prompt calls on two streams, a workspace each."""
    small = paged_case([(1, 3000 + 7 * r) for r in range(40)], 2, 128, 16, "e4m3", seed=17)
    large = paged_case([(500, 900), (300, 300)], 2, 128, 16, "bf16", seed=18)
    jobs = []
    for c in (small, large):
        q = _q(c, 8)
        want, _ = _run(c, q)
        g = dev(c)
        args, scales = cache_args(g)
        jobs.append((q.to(DEV), args, scales, max(n for n, _ in c["lengths"]), want, torch.cuda.Stream(), []))
    torch.cuda.synchronize()
    for _ in range(10):
        for q, args, scales, n, _, stream, outs in jobs:
            outs.append(glinattn_paged_attention(q, *args, **scales, max_q_len=n, stream=stream))
    torch.cuda.synchronize()
    for *_, want, _, outs in jobs:
        assert all(torch.equal(o, want) for o in outs)


def test_empty_batches_and_pools():
    """No request has tokens; no request has a cache; a pool without pages."""
    c = paged_case([(0, 20), (0, 0)], 1, 64, 16, "bf16", seed=19, num_tok=4)
    o = torch.full((4, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    got, status = _run(c, _q(c, 2), o=o, max_q_len=4)
    assert status == 0 and bool((got == 7).all())
    for n in (2, 100):
        q = torch.randn((n, 2, 64), device=DEV).to(torch.bfloat16)
        pool = torch.empty((0, 1, 16, 64), dtype=torch.bfloat16, device=DEV)
        table = torch.empty((1, 0), dtype=torch.int32, device=DEV)
        kv = torch.zeros(1, dtype=torch.int32, device=DEV)
        qs = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        assert bool((glinattn_paged_attention(q, pool, pool, table, kv, qs, max_q_len=n) == 0).all())


@pytest.mark.parametrize("R", [191, 192, 193, 400, 1500])
def test_more_requests_than_a_planning_pass_takes(R):
    c = paged_case([((r * 5) % 3, (r * 5) % 3 + (r * 11) % 40) for r in range(R)], 1, 64, 16, "bf16", seed=R)
    q = _q(c, 2)
    _check(c, q)
    _check(c, q, max_q_len=200)      # the kernel for many rows


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv,d", [(1, 1, 64), (2, 1, 128), (3, 1, 128), (8, 2, 64), (5, 1, 64), (12, 2, 128),
                                     (32, 1, 128), (33, 1, 64), (64, 1, 64), (100, 1, 128)])
def test_queries_of_others_do_not_matter(H, Hkv, d, cache):
    """The rows around a request hold other requests' queries, or none: NaN and infinities there."""
    c = paged_case([(150, 200), (7, 30), (130, 131), (1, 300), (64, 64)], Hkv, d, 16, cache, seed=H, first=2, num_tok=370)
    q = _q(c, H)
    want = torch.from_numpy(_check(c, q)).to(torch.bfloat16)
    start = c["q_start"].tolist()
    for r in range(len(c["lengths"])):
        mine = torch.zeros(c["num_tok"], dtype=torch.bool)
        mine[start[r]:start[r + 1]] = True
        bad = q.clone()
        bad[~mine] = torch.tensor([math.nan, math.inf, -math.inf])[torch.arange(int((~mine).sum())) % 3].to(torch.bfloat16)[:, None, None]
        got, status = _run(c, bad, o=torch.full_like(q, 7.0).to(DEV))
        assert status == 0 and torch.equal(got.cpu()[mine], want[mine])
        assert bool((got.cpu()[:2] == 7).all()) and bool((got.cpu()[start[-1]:] == 7).all())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv,d", [(4, 1, 128), (6, 2, 128), (2, 2, 64), (16, 1, 64)])
def test_many_short_prompts(H, Hkv, d, cache):
    """Several items per SM, most of them of a few cache tiles and with ragged ends."""
    c = paged_case([(1 + (r * 37) % 260, 1 + (r * 37) % 260 + (r * 53) % 150) for r in range(90)], Hkv, d, 16, cache, seed=H)
    q = _q(c, H)
    _check(c, q)
    first, _ = _run(c, q)
    for _ in range(10):
        again, status = _run(c, q)
        assert status == 0 and torch.equal(again, first)


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_below_kv_len_is_seen(d, cache, big):
    """A NaN element of a value row makes its channel NaN in every row that sees it, a NaN in a key every channel."""
    n = 150 if big else 3
    c = paged_case([(n, 200), (n, 200), (n, 160)], 1, d, 16, cache, seed=20)
    for r, (name, pos, ch) in enumerate([("v_cache", 20, d - 3), ("v_cache", 199 - n // 2, 5)]):
        c[name].view(torch.uint8 if cache == "e4m3" else torch.int16)[c["table"][r, pos // 16], 0, pos % 16, ch] = 0x7F if cache == "e4m3" else 0x7FC0
    c["k_cache"].view(torch.uint8 if cache == "e4m3" else torch.int16)[c["table"][2, 9], 0, 6, 1] = 0x7F if cache == "e4m3" else 0x7FC0
    got, status = _run(c, _q(c, 4))
    nan = got.float().isnan().cpu()
    assert status == 0
    assert bool(nan[:n, :, d - 3].all())
    assert bool(nan[2 * n - n // 2 - 1:2 * n, :, 5].all())
    rows = torch.arange(n) + 160 - n >= 150
    assert bool(nan[2 * n:][rows].all())
    assert int(nan[:n].sum()) == n * 4               # nothing else, where every row sees it


def test_max_q_len_of_zero():
    """Allowed where no request has new tokens; a request with some is refused."""
    c = paged_case([(0, 20), (0, 0)], 1, 64, 16, "bf16", seed=21, num_tok=3)
    o = torch.full((3, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    got, status = _run(c, _q(c, 2), o=o, max_q_len=0)
    assert status == 0 and bool((got == 7).all())
    c = paged_case([(0, 20), (3, 9)], 1, 64, 16, "bf16", seed=21)
    got, status = _run(c, _q(c, 2), o=o, max_q_len=0)
    assert status == DEV_BAD_COUNT and bool((got == 7).all())


@pytest.mark.parametrize("q_len,H,Hkv,d", [(1, 16, 4, 128), (1, 100, 1, 64), (5, 33, 3, 128), (9, 7, 7, 64), (257, 3, 1, 128)])
def test_every_row_of_a_shared_item_is_joined(q_len, H, Hkv, d):
    """Long caches cut into pieces, with row counts around the merge's own tiles."""
    c = paged_case([(q_len, 30000), (q_len, 17000)], Hkv, d, 64, "bf16", seed=22 + q_len)
    _check(c, _q(c, H))
