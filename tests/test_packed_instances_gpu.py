"""Kernel instances of the packed calls that need much work, or rows without alignment, to be chosen: the convolution's tiles
of 64 rows and the scan's pieces."""
import pytest
import torch

from test_scan_packed_gpu import case as scan_case, check as check_scan
from test_short_conv_gpu import case as conv_case, check as check_conv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")

# requests that begin and end at, before and behind multiples of 64, rows past a tile's end among them
ENDS = [63, 1, 64, 65, 0, 62, 2, 1, 127, 1, 0, 129, 3, 61, 191, 1, 1, 1, 126, 500, 12, 64, 64, 700, 3, 58]


@pytest.mark.parametrize("act,width", [(torch.bfloat16, 4), (torch.bfloat16, 2), (torch.float32, 4), (torch.float32, 3)])
@pytest.mark.parametrize("C,stride", [(9000, 0), (9004, 18016)])
def test_conv_tiles_of_64_rows(C, stride, act, width):
    c = conv_case(ENDS, C, width, act, seed=width, stride=stride, pad=3, first=2)
    assert c["x"].shape[0] * ((C + 31) // 32) // 4 // 64 >= 152 * 16
    some = [int(r % 3 != 1) for r in range(len(ENDS))]
    check_conv(c, resume=some)
    check_conv(c, silu=False, bias=False, resume=some, count=[n * (r % 4) // 3 if r % 4 < 3 else n for r, n in enumerate(ENDS)])
    check_conv(c, outputs=False, count=[min(n, 1 + r % 5) for r, n in enumerate(ENDS)])


LONG = [1500, 3, 0, 2049, 512, 513, 1024, 1025, 1, 1100]


@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,shift", [(33, 0), (40, 1), (7, 0)])
def test_scan_pieces_of_unaligned_rows(D, shift, act, N):
    """A number of channels that no vector fits, and slices whose base is off by one element."""
    c = scan_case(LONG, D, N, act, seed=N + D, strided=True, pad=3, first=2)
    if shift:
        for name in ("x", "z"):
            wide = torch.zeros((c[name].shape[0], D + 8), dtype=act, device=DEV)
            wide[:, shift:shift + D] = c[name]
            c[name] = wide[:, shift:shift + D]
        assert c["x"].data_ptr() % 16
    check_scan(c, resume=[int(r % 3 != 1) for r in range(10)])
    accept = [1500, 2, 0, 1537, 512, 0, 1000, 1025, 1, 512]
    y, pool = check_scan(c, count=accept)
    _, again = check_scan(c, count=accept, outputs=False)
    assert torch.equal(pool, again)
    check_scan(c, update=False, z=False, skip=False, out=torch.float32)
