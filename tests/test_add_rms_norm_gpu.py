"""GPU parity of glinattn_add_rms_norm with the fp64 oracle."""
import numpy as np
import pytest
import torch

from gated_deltanet_02_gb300 import glinattn_add_rms_norm
from oracle import layer_parts as L

from helpers import f64
from layer_parts_helpers import EPS32, HALF, check_e4m3, check_pow2_codes, close

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def _rel(width):
    """Relative error of a normed value in fp32: the sum of squares is added in chains of at most width / 512 + 80
    terms (32 of a thread and two trees, or every 512th element of a row), each addition and square off by 2^-24 and the
    root of the sum by half of that; then the sum's own roundings, root, quotient and two products."""
    return (0.5 * (width / 512 + 80) + 8) * EPS32


def _inputs(rows, width, act, res, seed=0, weight=True, stride=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, stride or width), generator=g).to(act).to(DEV)[:, :width]
    r = None if res is None else (torch.randn((rows, width), generator=g) * 3 + 1).to(res).to(DEV)
    w = (1 + 0.3 * torch.randn(width, generator=g)).to(DEV) if weight else None
    return x, r, w


def _check(x, r, w, got, eps=1e-6):
    y, out, scale = got
    width = x.shape[1]
    want, h = L.add_rms_norm(f64(x), f64(r), f64(w), eps)
    if r is not None:
        close(out, h, (HALF[r.dtype] + EPS32) * np.abs(h) + 1e-45, "sum")
    else:
        assert out is None
    rel = _rel(width)
    if y.dtype != E4M3:
        assert scale is None
        close(y, want, (HALF[y.dtype] + rel) * np.abs(want) + 1e-38, "y")
        return
    blocks = want.reshape(want.shape[0], scale.shape[1], -1)
    amax = np.abs(np.where(np.isfinite(blocks), blocks, 0.0)).max(-1)
    if scale.dtype == E8M0:
        code = scale.view(torch.uint8).cpu().numpy()
        check_pow2_codes(code, amax, rel)
        s = 2.0 ** (code.astype(np.float64) - 127)
    else:
        s = f64(scale)
        close(scale, np.maximum(amax / 448.0, 2.0 ** -100), rel * amax / 448.0 + 2.0 ** -123, "scale")
    check_e4m3(f64(y.float()).reshape(blocks.shape), s[..., None], blocks, rel * np.abs(blocks) + 1e-38)


@pytest.mark.parametrize("act,res", [(torch.bfloat16, None), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                     (torch.float32, torch.bfloat16), (torch.float32, torch.float32)])
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (5, 8), (130, 64), (9, 72), (4, 200), (3, 256), (7, 264), (2, 1001), (4, 2048),
                                        (3, 4104), (2, 8192), (2, 32768), (1, 40000)])
def test_norm(rows, width, act, res):
    x, r, w = _inputs(rows, width, act, res, seed=rows + width)
    for out in (torch.bfloat16, torch.float32):
        _check(x, r, w, glinattn_add_rms_norm(x, w, r, out_dtype=out))


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("rows,width", [(1, 128), (37, 256), (5, 384), (3, 2176), (2, 8192), (2, 33024)])
def test_e4m3(rows, width, group, pow2):
    for act, res in ((torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32), (torch.bfloat16, None)):
        x, r, w = _inputs(rows, width, act, res, seed=width + group)
        x[0, : min(width, 32)] = 0          # a block of zeros (where there is no residual)
        _check(x, r, w, glinattn_add_rms_norm(x, w, r, out_dtype=E4M3, group=group, scale_dtype=E8M0 if pow2 else None))


@pytest.mark.parametrize("rows,width,stride", [(5, 129, 129), (4, 256, 264), (6, 256, 257), (3, 96, 1001)])
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
def test_slices_and_odd_widths(rows, width, stride, act):
    x, r, w = _inputs(rows, width, act, act, seed=stride, stride=stride)
    _check(x, r, w, glinattn_add_rms_norm(x, w, r))
    _check(x, r, None, glinattn_add_rms_norm(x, None, r, out_dtype=E4M3))
    y = _inputs(rows, width, act, None, seed=stride, stride=stride + 1)[0][:, 1:]       # a base that is not 16-byte aligned
    _check(y, None, w[: width - 1].clone(), glinattn_add_rms_norm(y, w[: width - 1].clone()))
    if width % 32 == 0:
        _check(x, r, w, glinattn_add_rms_norm(x, w, r, out_dtype=E4M3, group=32, scale_dtype=E8M0))


@pytest.mark.parametrize("width", [7, 512, 4096, 40000])
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
def test_in_place(width, act):
    x, r, w = _inputs(6, width, act, act, seed=width)
    want, h = L.add_rms_norm(f64(x), f64(r), f64(w), 1e-6)
    x1, r1 = x.clone(), r.clone()
    y, out, _ = glinattn_add_rms_norm(x1, w, r1, residual_out=r1, y=x1)
    assert y is x1 and out is r1
    close(r1, h, (HALF[act] + EPS32) * np.abs(h), "sum")
    close(x1, want, (HALF[act] + _rel(width)) * np.abs(want), "y")
    x2 = x.clone()
    y2, out2, _ = glinattn_add_rms_norm(x2, w, r, residual_out=x2)      # the sum in x's place
    assert out2 is x2 and torch.equal(x2, r1) and torch.equal(y2, x1)


@pytest.mark.parametrize("width", [40, 100, 4096, 33000])
def test_sizes_of_values(width):
    """Rows of zeros, tiny and huge values (whose squares leave fp32), an infinity, NaN."""
    g = torch.Generator().manual_seed(width)
    x = torch.randn((7, width), generator=g)
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e30
    x[3] *= 1e37
    x[4, 3] = float("inf")
    x[5, 5] = float("nan")
    x, w = x.to(DEV), (1 + 0.1 * torch.randn(width, generator=g)).to(DEV)
    want, _ = L.add_rms_norm(f64(x), None, f64(w), 1e-6)
    assert np.isnan(want[4, 3]) and not want[4, 4]
    y, _, _ = glinattn_add_rms_norm(x, w)
    close(y, want, _rel(width) * np.abs(want) + 1e-38, "y")
    q, _, s = glinattn_add_rms_norm(x, w, out_dtype=E4M3)
    _check(x[:4], None, w, (q[:4], None, s[:4]))
    assert torch.isnan(q.float()[4, 3]) and not q.float()[4, 4] and bool(torch.isnan(q.float()[5]).all())
    assert s[0].item() == s[5].item() == 2.0 ** -100


def test_a_large_eps_and_no_weight():
    x, r, _ = _inputs(5, 300, torch.bfloat16, torch.float32, seed=2, weight=False)
    _check(x, r, None, glinattn_add_rms_norm(x, None, r, eps=10.0, out_dtype=torch.float32), eps=10.0)


def test_many_rows_pass_32_bit_offsets():
    """More than 2^31 elements: the last rows."""
    width = 4096
    rows = (1 << 31) // width + 3
    x = torch.zeros((rows, width), dtype=torch.bfloat16, device=DEV)
    x[-3:] = torch.randn((3, width), device=DEV).to(torch.bfloat16)
    y, out, s = glinattn_add_rms_norm(x, None, x, out_dtype=E4M3, group=128)
    _check(x[-3:], x[-3:], None, (y[-3:], out[-3:], s[-3:]))
    assert not bool(y[:-3].view(torch.uint8).any())


def test_no_rows():
    y, out, s = glinattn_add_rms_norm(torch.empty((0, 64), device=DEV), None, None, out_dtype=E4M3)
    assert y.shape == (0, 64) and out is None and s.shape == (0, 1)
