"""glinattn_add_rms_norm with e4m3 outputs and fp32 scales where factors could leave fp32: the smallest eps beside rows of
zeros and tiny values, large weights, outputs that overflow."""
import numpy as np
import pytest
import torch

from gated_deltanet_02_gb300 import glinattn_add_rms_norm
from oracle import layer_parts as L

from helpers import f64
from layer_parts_helpers import EPS32, check_e4m3, close

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
E4M3 = torch.float8_e4m3fn

# widths of each kernel: one, two and four chunks of 8 a thread, the scalar one; and rows whose base is not 16-byte aligned
WIDTHS = [(256, 0), (1024, 0), (4096, 0), (33024, 0), (256, 1), (4096, 1)]


def _rel(width):
    """Relative error of a normed value in fp32: chains of at most width / 512 + 80 additions of squares, halved by the
    root, and 8 roundings around it."""
    return (0.5 * (width / 512 + 80) + 8) * EPS32


def _rows(x, offset):
    """x in rows one element wider, from element `offset` on."""
    wide = torch.zeros((x.shape[0], x.shape[1] + 8 * offset), dtype=x.dtype)
    wide[:, offset:offset + x.shape[1]] = x
    return wide.to(DEV)[:, offset:offset + x.shape[1]]


def _check(x, r, w, group, eps):
    q, out, scale = glinattn_add_rms_norm(x, w, r, eps=eps, group=group, out_dtype=E4M3)
    width = x.shape[1]
    want, h = L.add_rms_norm(f64(x), f64(r), f64(w), eps)
    assert (np.abs(want) < 3e38).all()
    if r is not None:
        close(out, h, 2 * EPS32 * np.abs(h) + 1e-45, "sum")
    blocks = want.reshape(len(want), scale.shape[1], -1)
    amax = np.abs(blocks).max(-1)
    rel = _rel(width)
    # the scale: the maximum's error and the quotient's rounding, or its floor
    close(scale, np.maximum(amax / 448.0, 2.0 ** -100), (rel + EPS32) * amax / 448.0 + 2.0 ** -124, "scale")
    got = f64(q.float()).reshape(blocks.shape)
    check_e4m3(got, f64(scale)[..., None], blocks, rel * np.abs(blocks) + 1e-38)
    assert not got[blocks == 0].any()


@pytest.mark.parametrize("eps", [1e-20, 1e-17, 1e-6])
@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("width,offset", WIDTHS)
def test_zero_and_tiny_rows(width, offset, group, eps):
    """Rows of zeros give zeros at any eps; tiny rows, zeros among their elements, give their values."""
    g = torch.Generator().manual_seed(width + group)
    x = torch.randn((8, width), generator=g)
    for row, size in enumerate((0.0, 1e-38, 1e-37, 1e-35, 1e-28, 1e-19, 1e-9, 1.0)):
        x[row] *= size
    x[:, ::5] = 0
    x[6, :64] = 0                       # two blocks of zeros in a row of other values
    w = (1 + 0.1 * torch.randn(width, generator=g)).to(DEV)
    r = torch.randn((8, width), generator=g) * 1e-37
    r[0], r[:, ::5] = 0, 0
    _check(_rows(x, offset), None, w, group, eps)
    _check(_rows(x, offset), r.to(DEV), w, group, eps)
    bf = x.to(torch.bfloat16)
    _check(_rows(bf, offset), None, None, group, eps)


@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("width,offset", WIDTHS)
def test_large_and_small_weights(width, offset, group):
    """The product of a value and its weight may leave fp32 where the output does not."""
    g = torch.Generator().manual_seed(width)
    x = torch.randn((4, width), generator=g).clamp(-4, 4)
    x *= torch.tensor([1.0, 1e15, 1e-8, 1e30])[:, None]
    for size, eps in ((1e25, 1e-20), (1e37, 1e-6), (1e-25, 1e-20)):
        w = (size * (1 + 0.1 * torch.randn(width, generator=g).clamp(-3, 3))).to(DEV)
        _check(_rows(x, offset), None, w, group, eps)


@pytest.mark.parametrize("width,offset", WIDTHS)
def test_outputs_that_overflow(width, offset):
    """An output beyond fp32 counts as an infinity: +-448, and the scale is that of the finite ones."""
    x = torch.ones((2, width))
    x[0, 3], x[0, 7] = 8.0, -8.0
    x[1] *= 1e20
    w = torch.full((width,), 2e38 if width == 256 else 1e38)
    w[9] = 1e30
    want, _ = L.add_rms_norm(x.double().numpy(), None, w.double().numpy(), 1e-6)
    big = np.abs(want) > 4e38
    assert big[0].sum() == 2 and not big[1].any() and (np.abs(want[~big]) < 3e38).all()
    for group in (0, 32):
        q, _, scale = glinattn_add_rms_norm(_rows(x, offset), w.to(DEV), group=group, out_dtype=E4M3)
        got, s = f64(q.float()), f64(scale)
        assert np.array_equal(got[big], [448.0, -448.0])
        amax = np.where(big, 0.0, np.abs(want)).reshape(2, s.shape[1], -1).max(-1)
        close(scale, amax / 448.0, (_rel(width) + EPS32) * amax / 448.0, "scale")
        each = np.repeat(s, width // s.shape[1], 1)
        check_e4m3(got[~big], each[~big], want[~big], _rel(width) * np.abs(want[~big]) + 1e-38)
