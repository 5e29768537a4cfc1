"""Arguments of the paged attention at the ends of their ranges, without a GPU."""
import ctypes

import pytest
import torch

from gated_deltanet_02_gb300 import glinattn as G
from gated_deltanet_02_gb300 import glinattn_paged_attention

A = 0x10000
INVALID = 1


def _args(**kw):
    base = dict(cache_dtype=G.BF16, num_req=2, num_tok=4, heads=4, kv_heads=2, head_dim=128, page_size=16, num_pages=8,
                max_pages=4, max_q_len=2, scale=0.1, q=A, k_cache=3 * A, v_cache=4 * A, page_table=5 * A, kv_len=6 * A,
                q_start=7 * A, o=8 * A, workspace=16 * A, workspace_bytes=1 << 40)
    base.update(kw)
    return G.PagedAttnArgs(**base)


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38])
def test_a_scale_that_overflows_in_log2_units_is_refused(scale):
    assert G.library().glinattn_paged_attention(ctypes.byref(_args(scale=scale)), None) == INVALID
    assert G.library().glinattn_paged_attention_workspace_size(ctypes.byref(_args(scale=scale))) == 0
    assert G.library().glinattn_paged_attention_workspace_size(ctypes.byref(_args(scale=2.3e38))) > 0


@pytest.mark.parametrize("n", [1 << 31, 1 << 32, (1 << 32) + 1, -1])
def test_max_q_len_past_32_bits_is_refused(n):
    """Not cut to its low bits, which would skip requests or select another kernel."""
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    cache = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="max_q_len"):
        glinattn_paged_attention(torch.zeros(3, 4, 64, dtype=torch.bfloat16), cache, cache, i(2, 3), i(2), i(3), max_q_len=n)
