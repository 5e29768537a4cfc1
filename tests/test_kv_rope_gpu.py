"""GPU parity of glinattn_kv_append_rope with the fp64 oracle."""
import numpy as np
import pytest
import torch

from gated_deltanet_02_gb300 import glinattn_kv_append, glinattn_kv_append_rope
from gated_deltanet_02_gb300.glinattn import DEV_BAD_COUNT, DEV_BAD_SLOT
from oracle import layer_parts as L
from oracle import paged as P

from helpers import f64
from layer_parts_helpers import EPS32, HALF, check_e4m3, check_pow2_codes, close
from paged_helpers import cache_args, dev, paged_case

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
MARK = 7.0
BF16 = torch.bfloat16

LENGTHS = {
    "one": [(1, 1)], "mixed": [(1, 40), (0, 7), (17, 17), (3, 130), (0, 0), (33, 95)], "short": [(5, 3), (2, 0), (4, 200)],
    "many": [(1, 1 + 13 * r) for r in range(70)], "search": [((r * 7) % 3, (r * 7) % 3 + r % 50) for r in range(1100)],
}


def freqs(rot, base=10000.0):
    return torch.from_numpy(base ** (-np.arange(0, rot, 2) / rot)).float()


def new_rows(c, H, seed, fused=False):
    g = torch.Generator().manual_seed(seed)
    n, k, d = c["num_tok"], c["Hkv"], c["d"]
    rows = torch.randn((n, H + 2 * k, d), generator=g).to(BF16).to(DEV)
    parts = rows[:, :H], rows[:, H:H + k], rows[:, H + k:]
    return parts if fused else tuple(p.contiguous() for p in parts)


def check(c, q, k, v, inv, interleaved=False, scale=1.0, status=0, in_place=False):
    g = dev(c)
    args, kw = cache_args(g)
    before = {name: g[name].clone() for name in ("k_cache", "v_cache")}
    codes = {name: None if g[name] is None else g[name].clone() for name in ("k_scale", "v_scale")}
    qd, kd, vd = f64(q), f64(k), f64(v)
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = q if in_place else torch.full(q.shape, MARK, dtype=BF16, device=DEV)
    got, *_ = glinattn_kv_append_rope(q, k, v, inv.to(DEV), *args, interleaved=interleaved, rope_scale=scale, q_out=out, dev_status=word, **kw)
    assert got is out and int(word.item()) == status
    # sine and cosine to 4 units of 2^-24, three roundings of products and sum, the scale's
    rel = 8 * EPS32
    q_want = qd.copy() if in_place else np.full(qd.shape, MARK)
    q_tol = np.zeros(qd.shape)
    written = []
    for r in range(len(c["lengths"])):
        for i, pos in P.positions(c["q_start"], c["kv_len"], r):
            s0, s1, kv = int(c["q_start"][r]), int(c["q_start"][r + 1]), int(c["kv_len"][r])
            if pos < 0 or s0 < 0 or s1 > c["num_tok"] or not 0 <= kv <= c["table"].shape[1] * c["page"]:
                continue
            q_want[i:i + 1], size = L.rotate(qd[i:i + 1], [pos], f64(inv), interleaved, scale)
            q_tol[i:i + 1] = rel * size + HALF[BF16] * np.abs(q_want[i:i + 1]) + 1e-39
            pg = int(c["table"][r, pos // c["page"]])
            if 0 <= pg < c["pages"]:
                written.append((i, pos, pg, pos % c["page"]))
    close(out, q_want, q_tol, "q")
    i, pos, pg, at = (np.array([w[j] for w in written], dtype=np.int64) for j in range(4))
    keep = np.ones((c["pages"], c["page"]), bool)
    keep[pg, at] = False
    for name, x in (("k", kd), ("v", vd)):
        cache = g[name + "_cache"].float().cpu().double().numpy()
        old = before[name + "_cache"].float().cpu().double().numpy()
        assert np.array_equal(cache.transpose(0, 2, 1, 3)[keep], old.transpose(0, 2, 1, 3)[keep]), name
        if not written:
            continue
        want, size = L.rotate(x[i], pos, f64(inv), interleaved, scale) if name == "k" else (x[i], np.zeros_like(x[i]))
        rows = cache[pg, :, at]
        if c["cache"] == "bf16":
            close(rows, want, rel * size + (HALF[BF16] * np.abs(want) + 1e-39 if name == "k" else 0.0), name)
        else:
            code = g[name + "_scale"].cpu().numpy()
            assert np.array_equal(code.transpose(0, 2, 1)[keep], codes[name + "_scale"].cpu().numpy().transpose(0, 2, 1)[keep])
            code = code[pg, :, at]
            top = np.abs(want).argmax(-1)[..., None]
            amax = np.take_along_axis(np.abs(want), top, -1)[..., 0]
            check_pow2_codes(code, amax, 2 * rel * (size.max() / max(amax.min(), 1e-30) if name == "k" else 0.0))
            check_e4m3(rows, (2.0 ** (code.astype(np.float64) - 127))[..., None], want, rel * size)
    return g, out


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H,Hkv,d,page,rot", [(1, 1, 64, 16, 64), (6, 3, 128, 32, 128), (16, 8, 128, 64, 48), (5, 2, 64, 128, 16), (2, 1, 128, 16, 112)])
@pytest.mark.parametrize("name", list(LENGTHS))
def test_rotated_append(name, H, Hkv, d, page, rot, interleaved, cache):
    if name == "search" and page != 16:
        pytest.skip("one page size for the large batch")
    c = paged_case(LENGTHS[name], Hkv, d, page, cache, seed=3)
    check(c, *new_rows(c, H, 4, fused=rot == d), freqs(rot), interleaved, 1.0 if interleaved else 1.25)


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_on_slices(interleaved):
    c = paged_case(LENGTHS["mixed"], 2, 128, 16, "bf16", seed=5)
    check(c, *new_rows(c, 6, 6, fused=True), freqs(128), interleaved, in_place=True)


def test_far_positions():
    """Angles of positions past a hundred million: the fraction of a turn is exact."""
    page, n = 128, 3
    max_pages = 1 << 20
    table = torch.full((1, max_pages), -1, dtype=torch.int32, device=DEV)
    pos = 134217000
    table[0, pos // page] = 1
    kc = torch.zeros((2, 1, page, 64), dtype=BF16, device=DEV)
    vc = torch.zeros_like(kc)
    kv, qs = torch.tensor([pos + n], dtype=torch.int32, device=DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(7)
    q, k = (torch.randn((n, 1, 64), generator=g).to(BF16).to(DEV) for _ in range(2))
    inv = freqs(64)
    inv[3], inv[4] = -0.7, 12345.678
    out, _, _ = glinattn_kv_append_rope(q, k, k, inv.to(DEV), kc, vc, table, kv, qs)
    assert pos % page + n <= page
    want, size = L.rotate(f64(q), pos + np.arange(n), f64(inv))
    # the oracle's extended precision keeps 2^-64 of angles up to 2^41
    close(out, want, (8 * EPS32 + 2.0 ** -22) * size + HALF[BF16] * np.abs(want))
    wk, size = L.rotate(f64(k), pos + np.arange(n), f64(inv))
    close(kc[1, 0, pos % page:pos % page + n], wk[:, 0], (8 * EPS32 + 2.0 ** -22) * size[:, 0] + HALF[BF16] * np.abs(wk[:, 0]))


def test_frequencies_of_every_size():
    """Powers of two from the smallest subnormal to 2^23 turn as they should; larger ones and NaN give NaN."""
    inv = torch.tensor([2.0 ** e for e in range(-31, 24)] + [0.0, -0.0, 2.0 ** -149, 2.0 ** -126, -3.0, 1e-20, 0.1, 2.0 ** 24, float("nan")])
    assert len(inv) == 64
    c = paged_case([(9, 1000), (3, 5)], 1, 128, 16, "bf16", seed=8)
    q, k, v = new_rows(c, 1, 9)
    g = dev(c)
    args, kw = cache_args(g)
    out, _, _ = glinattn_kv_append_rope(q, k, v, inv.to(DEV), *args, **kw)
    pos = np.concatenate([np.arange(991, 1000), np.arange(2, 5)])
    fine = np.r_[0:62, 64:126]
    with np.errstate(invalid="ignore"):
        want, size = L.rotate(f64(q), pos, f64(inv))
    assert bool(torch.isnan(out[..., [62, 63, 126, 127]]).all())
    close(out[..., fine], want[..., fine], (8 * EPS32 + 2.0 ** -22) * size[..., fine] + HALF[BF16] * np.abs(want[..., fine]))


def test_zero_frequencies_are_the_plain_append():
    """Without any turn the cache is glinattn_kv_append's, bit for bit, infinities and NaN too."""
    for cache in ("bf16", "e4m3"):
        c = paged_case(LENGTHS["mixed"], 3, 64, 16, cache, seed=10)
        q, k, v = new_rows(c, 3, 11)
        v[1::7, -1, 3], v[2::7, 0, 5], v[::5, 1] = float("inf"), float("nan"), 0.0
        a, b = dev(c), dev(c)
        (args, kw), (args2, kw2) = cache_args(a), cache_args(b)
        out, _, _ = glinattn_kv_append_rope(q, k, v, torch.zeros(32, device=DEV), *args, **kw)
        glinattn_kv_append(k, v, *args2, **kw2)
        assert torch.equal(out[:1], q[:1])
        for name in ("k_cache", "v_cache"):
            assert torch.equal(a[name].view(torch.uint8), b[name].view(torch.uint8)), name
        for name in ("k_scale", "v_scale"):
            assert a[name] is None or torch.equal(a[name], b[name])


def test_keys_and_values_alone():
    c = paged_case([(4, 20)], 2, 64, 16, "bf16", seed=12)
    q, k, v = new_rows(c, 2, 13)
    a, b = dev(c), dev(c)
    (args, kw), (args2, kw2) = cache_args(a), cache_args(b)
    out, _, _ = glinattn_kv_append_rope(None, k, v, freqs(64).to(DEV), *args, **kw)
    glinattn_kv_append_rope(q, k, v, freqs(64).to(DEV), *args2, **kw2)
    assert out is None and torch.equal(a["k_cache"], b["k_cache"]) and torch.equal(a["v_cache"], b["v_cache"])


def test_padded_batch_and_rows_before_the_first_request():
    c = paged_case([(3, 20), (2, 9)], 2, 128, 16, "e4m3", seed=14, num_tok=12, first=2)
    check(c, *new_rows(c, 4, 15), freqs(128))


def test_bad_pages_and_lengths_are_flagged_and_skipped():
    c = paged_case([(2, 20), (2, 20), (2, 20), (2, 20)], 1, 64, 16, "bf16", seed=16)
    c["table"][1, 1] = c["pages"]
    c["kv_len"][2] = 1000
    check(c, *new_rows(c, 2, 17), freqs(64), status=DEV_BAD_SLOT | DEV_BAD_COUNT)


def test_far_pages_pass_32_bit_offsets():
    page, Hkv, d = 128, 8, 128
    pages = (1 << 32) // (page * Hkv * d * 2) + 2
    kc = torch.zeros((pages, Hkv, page, d), dtype=BF16, device=DEV)
    vc = torch.zeros_like(kc)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device=DEV)
    kv, qs = torch.tensor([5], dtype=torch.int32, device=DEV), torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(18)
    k, v = (torch.randn((5, Hkv, d), generator=g).to(BF16).to(DEV) for _ in range(2))
    glinattn_kv_append_rope(None, k, v, freqs(128).to(DEV), kc, vc, table, kv, qs)
    want, size = L.rotate(f64(k), np.arange(5), f64(freqs(128)))
    close(kc[-1, :, :5].transpose(0, 1), want, 8 * EPS32 * size + HALF[BF16] * np.abs(want))
    assert torch.equal(vc[-1, :, :5].transpose(0, 1), v) and not bool(kc[:-1].any()) and not bool(kc[-1, :, 5:].any())
