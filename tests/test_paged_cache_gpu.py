"""GPU parity of glinattn_kv_append and glinattn_kv_gather with the oracle:
stored values, scales and rows read back are compared bit for bit."""
import numpy as np
import pytest
import torch

from gated_deltanet_02_gb300 import glinattn_kv_append, glinattn_kv_gather
from gated_deltanet_02_gb300.glinattn import DEV_BAD_COUNT, DEV_BAD_SLOT
from oracle import paged as P

from paged_helpers import cache_args, dev, paged_case, rows_of

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")

LENGTHS = [
    [(1, 1)],
    [(1, 40), (0, 7), (17, 17), (3, 130), (0, 0), (33, 95)],
    [(5, 3), (2, 0), (4, 200)],                        # more new tokens than positions
    [(1, 1 + 13 * r) for r in range(70)],              # more requests than a warp has lanes
    [((r * 7) % 3, (r * 7) % 3 + r % 50) for r in range(1100)],  # three rounds of the request search
]


def _new(c, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        x = torch.randn((c["num_tok"], c["Hkv"], c["d"]), generator=g)
        if kind == "wide":  # every exponent that bf16 has, rows of zeros, infinities, NaN
            x = x * 2.0 ** torch.randint(-130, 128, (c["num_tok"], c["Hkv"], 1), generator=g).double()
            x[::5, 0] = 0.0
            x[1::7, -1, 3] = float("inf")
            x[2::7, -1, 5] = -float("inf")
            x[3::7, 0, 7] = float("nan")
        out.append(x.float().to(torch.bfloat16))
    return out


def _expected(c, new):
    """The whole cache after the append, as values and exponents."""
    out = {}
    for name, x in zip(("k", "v"), new):
        val = c[name + "_cache"].float().double().numpy().copy()
        code = None if c["cache"] == "bf16" else c[name + "_scale"].numpy().copy()
        xs = x.double().numpy()
        for r in range(len(c["lengths"])):
            for i, pos in P.positions(c["q_start"], c["kv_len"], r):
                if pos < 0:
                    continue
                pg, row = int(c["table"][r, pos // c["page"]]), pos % c["page"]
                if c["cache"] == "bf16":
                    val[pg, :, row] = xs[i]
                else:
                    v, e = P.quantise(xs[i])
                    val[pg, :, row], code[pg, :, row] = v, e + 127
        out[name] = (val, code)
    return out


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hkv,d,page", [(1, 64, 16), (3, 128, 32), (8, 128, 64), (2, 64, 128)])
@pytest.mark.parametrize("lengths", LENGTHS, ids=["one", "mixed", "short", "many", "search"])
def test_append_then_gather(lengths, Hkv, d, page, cache):
    if len(lengths) > 1000 and page != 16:
        pytest.skip("one page size for the large batch")
    c = paged_case(lengths, Hkv, d, page, cache, seed=3)
    new = _new(c, 4, "wide")
    g = dev(c)
    args, kw = cache_args(g)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    glinattn_kv_append(new[0].to(DEV), new[1].to(DEV), *args, **kw, dev_status=status)
    want = _expected(c, new)
    for name in ("k", "v"):
        val, code = want[name]
        assert np.array_equal(g[name + "_cache"].float().cpu().double().numpy(), val, equal_nan=True), name
        if code is not None:
            assert np.array_equal(g[name + "_scale"].cpu().numpy(), code), name
    # the way back: the rows of the same tokens; those at negative positions stay as they were
    k = torch.full((c["num_tok"], Hkv, d), 7.0, dtype=torch.bfloat16, device=DEV)
    v = torch.full_like(k, 7.0)
    glinattn_kv_gather(*args, k=k, v=v, **kw, dev_status=status)
    for name, got in (("k", k), ("v", v)):
        val, code = want[name]
        ref = np.full((c["num_tok"], Hkv, d), 7.0)
        for r in range(len(lengths)):
            for i, pos in P.positions(c["q_start"], c["kv_len"], r):
                if pos >= 0:
                    pg, row = int(c["table"][r, pos // page]), pos % page
                    ref[i] = val[pg, :, row] if code is None else val[pg, :, row] * 2.0 ** (code[pg, :, row].astype(np.float64) - 127)[:, None]
        assert np.array_equal(got.double().cpu().numpy(), ref, equal_nan=True), name
    assert int(status.item()) == 0


def test_gather_reads_whole_prefixes():
    c = paged_case([(0, 130), (0, 1), (0, 0), (0, 77)], 2, 64, 32, "e4m3", seed=9)
    g = dev(c)
    args, kw = cache_args(g)
    start = torch.tensor(np.concatenate([[0], np.cumsum([kv for _, kv in c["lengths"]])]), dtype=torch.int32, device=DEV)
    k, v = glinattn_kv_gather(*args[:4], start, num_tok=int(start[-1]), **kw)
    for name, got in (("k", k), ("v", v)):
        assert np.array_equal(got.double().cpu().numpy(), np.concatenate(rows_of(c, name)))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_padded_batch_and_rows_before_the_first_request(cache):
    c = paged_case([(3, 20), (2, 9)], 2, 128, 16, cache, seed=5, num_tok=12, first=2)
    new = _new(c, 6)
    g = dev(c)
    args, kw = cache_args(g)
    glinattn_kv_append(new[0].to(DEV), new[1].to(DEV), *args, **kw)
    want = _expected(c, new)
    assert np.array_equal(g["k_cache"].float().cpu().double().numpy(), want["k"][0])
    k = torch.full((12, 2, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    glinattn_kv_gather(*args, k=k, v=k.clone(), **kw)
    assert bool((k[:2] == 7).all()) and bool((k[7:] == 7).all()) and not bool((k[2:7] == 7).any())


def test_bad_pages_and_lengths_are_flagged_and_skipped():
    c = paged_case([(2, 20), (2, 20), (2, 20), (2, 20)], 1, 64, 16, "bf16", seed=7)
    new = _new(c, 8)
    c["table"][1, 1] = c["pages"]        # request 1: the page of its new tokens is past the pool
    c["kv_len"][2] = 1000                # request 2: longer than its page table
    g = dev(c)
    args, kw = cache_args(g)
    before = g["k_cache"].clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    glinattn_kv_append(new[0].to(DEV), new[1].to(DEV), *args, **kw, dev_status=status)
    assert int(status.item()) == DEV_BAD_SLOT | DEV_BAD_COUNT
    got, x = g["k_cache"].cpu(), new[0]
    for r in (0, 3):
        pg = int(c["table"][r, 1])
        assert torch.equal(got[pg, 0, 2], x[2 * r, 0]) and torch.equal(got[pg, 0, 3], x[2 * r + 1, 0])
    changed = (got != before.cpu()).flatten(1).any(1).nonzero().flatten().tolist()
    assert sorted(changed) == sorted(int(c["table"][r, 1]) for r in (0, 3))
    k = torch.full((8, 1, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    glinattn_kv_gather(*args, k=k, v=k.clone(), **kw)
    assert bool((k[2:6] == 7).all()) and torch.equal(k[:2].cpu(), x[:2]) and torch.equal(k[6:].cpu(), x[6:])


def test_far_pages_pass_32_bit_offsets():
    """A pool of more than 2^32 bytes: the last page's rows."""
    page, Hkv, d = 128, 8, 128
    pages = (1 << 32) // (page * Hkv * d * 2) + 2
    kc = torch.zeros((pages, Hkv, page, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device=DEV)
    kv, qs = torch.tensor([5], dtype=torch.int32, device=DEV), torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    k = torch.randn((5, Hkv, d), device=DEV).to(torch.bfloat16)
    v = torch.randn((5, Hkv, d), device=DEV).to(torch.bfloat16)
    glinattn_kv_append(k, v, kc, vc, table, kv, qs)
    assert torch.equal(kc[-1, :, :5].transpose(0, 1), k) and torch.equal(vc[-1, :, :5].transpose(0, 1), v)
    assert not bool(kc[-1, :, 5:].any())
    k2, v2 = glinattn_kv_gather(kc, vc, table, kv, qs, num_tok=5)
    assert torch.equal(k2, k) and torch.equal(v2, v)


@pytest.mark.parametrize("d,Hkv,page", [(64, 1, 16), (64, 3, 32), (128, 2, 16), (128, 1, 128)])
def test_gather_of_many_rows(d, Hkv, page):
    """A warp's rows that go on in a page, into the next one and into another request; rows at negative positions,
    in no request, behind a bad page and of a request that is out of bounds stay as they were."""
    c = paged_case([(2, 300), (4001, 4001), (0, 5), (7, 3), (1, 9), (1, 900), (1, 33), (2700, 5003), (50, 60), (1500, 1700)],
                   Hkv, d, page, "e4m3", seed=d, num_tok=8300, first=3)
    g = dev(c)
    bad_page, bad_len = 7, 8                            # requests
    g["table"][bad_page, 3000 // page] = c["pages"]
    g["kv_len"][bad_len] = -1
    args, kw = cache_args(g)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = [torch.full((c["num_tok"], Hkv, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    glinattn_kv_gather(*args, k=out[0], v=out[1], dev_status=status, **kw)
    assert int(status.item()) == DEV_BAD_SLOT | DEV_BAD_COUNT
    for x, name in zip(out, ("k", "v")):
        want = np.full((c["num_tok"], Hkv, d), 7.0)
        for r, rows in enumerate(rows_of(c, name)):
            for i, pos in P.positions(c["q_start"], c["kv_len"], r):
                if pos >= 0 and r != bad_len and not (r == bad_page and pos // page == 3000 // page):
                    want[i] = rows[pos]
        assert np.array_equal(x.float().cpu().double().numpy(), want)
