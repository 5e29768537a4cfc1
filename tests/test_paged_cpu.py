"""The paged-cache, attention and acceptance calls without a GPU: struct
layout, refusals of the C ABI and of the binding, and the oracle's own pins."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from gated_deltanet_02_gb300 import (glinattn_accept_drafts, glinattn_kv_append, glinattn_kv_gather,
                                     glinattn_paged_attention)
from gated_deltanet_02_gb300 import glinattn as G
from oracle import paged as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000
INVALID, UNSUPPORTED = 1, 2


def test_struct_layout_matches_header(tmp_path):
    structs = ((G.KvArgs, "glinattn_kv_args"), (G.PagedAttnArgs, "glinattn_paged_attn_args"),
               (G.AcceptArgs, "glinattn_accept_args"))
    src = tmp_path / "layout.c"
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "glinattn.h"', "int main(void){"]
    for ct, name in structs:
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f}));' for f, _ in ct._fields_]
    src.write_text("\n".join(lines + ["return 0;}"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for ct, _ in structs:
        want.append(ctypes.sizeof(ct))
        want += [getattr(ct, f).offset for f, _ in ct._fields_]
    assert got == want


def _kv(**kw):
    base = dict(cache_dtype=G.BF16, num_req=2, num_tok=4, kv_heads=2, head_dim=128, page_size=16, num_pages=8,
                max_pages=4, k=A, v=2 * A, k_cache=3 * A, v_cache=4 * A, page_table=5 * A, kv_len=6 * A, q_start=7 * A)
    base.update(kw)
    return G.KvArgs(**base)


def _attn(**kw):
    base = dict(cache_dtype=G.BF16, num_req=2, num_tok=4, heads=4, kv_heads=2, head_dim=128, page_size=16, num_pages=8,
                max_pages=4, max_q_len=2, scale=0.1, q=A, k_cache=3 * A, v_cache=4 * A, page_table=5 * A, kv_len=6 * A,
                q_start=7 * A, o=8 * A, workspace=16 * A, workspace_bytes=1 << 40)
    base.update(kw)
    return G.PagedAttnArgs(**base)


def _acc(**kw):
    base = dict(num_req=2, draft_len=3, vocab=100, target_probs=A, draft_probs=2 * A, draft_tokens=3 * A, uniforms=4 * A,
                accept=5 * A, tokens=6 * A)
    base.update(kw)
    return G.AcceptArgs(**base)


CACHE = [
    (dict(cache_dtype=G.F32), INVALID), (dict(cache_dtype=9), INVALID), (dict(num_req=-1), INVALID),
    (dict(num_req=65537), INVALID), (dict(num_tok=-1), INVALID), (dict(kv_heads=0), INVALID),
    (dict(num_pages=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(max_pages=1 << 29), INVALID),
    (dict(num_pages=1 << 30), INVALID), (dict(head_dim=0), INVALID), (dict(head_dim=96), UNSUPPORTED),
    (dict(head_dim=256), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=0), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID),
    (dict(k_cache=3 * A + 8), INVALID), (dict(page_table=None), INVALID), (dict(page_table=5 * A + 2), INVALID),
    (dict(kv_len=None), INVALID), (dict(q_start=None), INVALID), (dict(cache_dtype=G.E4M3), INVALID),
    (dict(cache_dtype=G.E4M3, k_scale=9 * A), INVALID), (dict(cache_dtype=G.E4M3, k_scale=9 * A, v_scale=9 * A + 1), INVALID),
]


@pytest.mark.parametrize("kw,code", CACHE + [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=A + 8), INVALID)])
@pytest.mark.parametrize("name", ["glinattn_kv_append", "glinattn_kv_gather"])
def test_cache_call_refusals(name, kw, code):
    assert getattr(G.library(), name)(ctypes.byref(_kv(**kw)), None) == code


@pytest.mark.parametrize("kw,code", CACHE + [
    (dict(heads=514), UNSUPPORTED), (dict(heads=3), INVALID), (dict(heads=0), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID), (dict(max_q_len=-1), INVALID),
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(q=A + 2), INVALID), (dict(o=A + 4), INVALID),
    (dict(num_tok=1 << 30), INVALID), (dict(workspace=None), INVALID), (dict(workspace_bytes=64), INVALID),
    (dict(workspace=16 * A + 8), INVALID), (dict(max_q_len=100, workspace_bytes=1 << 20), INVALID)])
def test_attention_refusals(kw, code):
    assert G.library().glinattn_paged_attention(ctypes.byref(_attn(**kw)), None) == code


@pytest.mark.parametrize("kw", [
    dict(num_req=-1), dict(draft_len=-1), dict(draft_len=1025), dict(vocab=0), dict(vocab=(1 << 22) + 1),
    dict(target_probs=None), dict(uniforms=None), dict(accept=None), dict(tokens=None), dict(draft_tokens=None),
    dict(target_probs=A + 2), dict(tokens=A + 1)])
def test_accept_refusals(kw):
    assert G.library().glinattn_accept_drafts(ctypes.byref(_acc(**kw)), None) == INVALID


def test_null_structs_and_empty_calls():
    lib = G.library()
    for name in ("glinattn_kv_append", "glinattn_kv_gather", "glinattn_paged_attention", "glinattn_accept_drafts"):
        assert getattr(lib, name)(None, None) == INVALID
    assert lib.glinattn_kv_append(ctypes.byref(_kv(num_tok=0, k=None, v=None)), None) == 0
    assert lib.glinattn_kv_gather(ctypes.byref(_kv(num_req=0)), None) == 0
    assert lib.glinattn_paged_attention(ctypes.byref(_attn(num_tok=0, q=None, o=None)), None) == 0
    assert lib.glinattn_accept_drafts(ctypes.byref(_acc(num_req=0)), None) == 0


def test_workspace_size_goes_by_sizes_alone():
    lib = G.library()
    size = lambda **kw: lib.glinattn_paged_attention_workspace_size(ctypes.byref(_attn(**kw)))  # noqa: E731
    few, many = size(max_q_len=1), size(max_q_len=1000)
    assert 0 < few < many < 1 << 27
    assert size(max_q_len=1, num_req=200, num_tok=200, max_pages=4096) == few
    assert size(num_tok=0) == 0 and size(num_req=0) == 0 and size(head_dim=96) == 0


def _cache(P_=4, H=2, page=16, d=64, dtype=torch.bfloat16):
    return torch.zeros(P_, H, page, d).to(dtype)


def _i(*s):
    return torch.zeros(*s, dtype=torch.int32)


def test_binding_refusals():
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    ok = (_cache(), _cache(), _i(2, 3), _i(2), _i(3))
    sc = torch.zeros(4, 2, 16, dtype=torch.uint8)
    with pytest.raises(TypeError):   # k in another dtype
        glinattn_kv_append(k.float(), k, *ok)
    with pytest.raises(ValueError):  # heads of k and cache differ
        glinattn_kv_append(k[:, :1].contiguous(), k, *ok)
    with pytest.raises(ValueError):  # a strided k
        glinattn_kv_append(k.transpose(0, 1).contiguous().transpose(0, 1), k, *ok)
    with pytest.raises(TypeError):   # a cache dtype that is not built
        glinattn_kv_append(k, k, _cache(dtype=torch.float16), _cache(dtype=torch.float16), *ok[2:])
    with pytest.raises(ValueError):  # e4m3 without scales
        glinattn_kv_append(k, k, _cache(dtype=torch.float8_e4m3fn), _cache(dtype=torch.float8_e4m3fn), *ok[2:])
    with pytest.raises(ValueError):  # scales with bf16
        glinattn_kv_append(k, k, *ok, k_scale=sc, v_scale=sc)
    with pytest.raises(ValueError):  # scales of the wrong shape
        glinattn_kv_gather(_cache(dtype=torch.float8_e4m3fn), _cache(dtype=torch.float8_e4m3fn), *ok[2:], num_tok=1,
                           k_scale=sc[:3], v_scale=sc)
    with pytest.raises(ValueError):  # q_start is [R + 1]
        glinattn_kv_append(k, k, *ok[:4], _i(2))
    with pytest.raises(TypeError):   # lengths are int32
        glinattn_kv_append(k, k, *ok[:3], _i(2).long(), _i(3))
    with pytest.raises(ValueError):  # neither num_tok nor outputs
        glinattn_kv_gather(*ok)
    with pytest.raises(ValueError):  # o of another shape
        glinattn_paged_attention(torch.zeros(3, 4, 64, dtype=torch.bfloat16), *ok, o=k)
    with pytest.raises(TypeError):   # q must be bf16
        glinattn_paged_attention(torch.zeros(3, 4, 64), *ok)
    with pytest.raises(ValueError):  # host tensors
        glinattn_kv_append(k, k, *ok)
    t, u = torch.zeros(2, 3, 10), torch.zeros(2, 3)
    with pytest.raises(ValueError):  # draft rows: one fewer than target rows
        glinattn_accept_drafts(t, t, _i(2, 2), u)
    with pytest.raises(TypeError):   # tokens are int32
        glinattn_accept_drafts(t, None, _i(2, 2).long(), u)
    with pytest.raises(ValueError):  # uniforms [R, D + 1]
        glinattn_accept_drafts(t, None, _i(2, 2), u[:, :2].contiguous())
    with pytest.raises(TypeError):   # probabilities are fp32
        glinattn_accept_drafts(t.double(), None, _i(2, 2), u)


# ---- the oracle ----------------------------------------------------------------

def test_oracle_e4m3_rounding_matches_torch():
    x = torch.cat([torch.linspace(-448, 448, 20001), torch.linspace(-0.1, 0.1, 20001)])
    assert np.array_equal(P.round_e4m3(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("a,e", [(448.0, 0), (449.0, 1), (224.0, -1), (225.0, 0), (1.0, -8), (1.75, -8), (1.7578125, -7),
                                 (0.0, -100), (3.0e38, 119), (2.9e38, 119), (1e-38, -100)])
def test_oracle_scale_exponent(a, e):
    assert P.scale_exponent(np.array([0.0, -a, a / 3, np.nan, np.inf])) == e


def test_oracle_attention_is_softmax():
    g = np.random.default_rng(0)
    q, k, v = g.normal(size=(3, 2, 8)), g.normal(size=(5, 1, 8)), g.normal(size=(5, 1, 8))
    o, _ = P.attention(q, [k], [v], [0, 3], [5], 0.5)
    for i in range(3):
        w = torch.softmax(torch.from_numpy(0.5 * k[:3 + i, 0] @ q[i, 1]), -1).numpy()
        assert np.allclose(o[i, 1], w @ v[:3 + i, 0], rtol=1e-12)


def test_oracle_accept_by_hand():
    target = np.array([[[0.5, 0.5, 0.0], [0.25, 0.25, 0.5]]], np.float32)
    draft = np.array([[[0.25, 0.75, 0.0]]], np.float32)
    u = np.array([[0.6, 0.5]], np.float32)
    a, t = P.accept_drafts(target, draft, np.array([[1]], np.int32), u)   # 0.6 * 0.75 < 0.5: accepted, then the median
    assert a[0] == 1 and t.tolist() == [[1, 2]]
    u[0, 0] = 0.7                                                          # rejected: the residual is all on token 0
    a, t = P.accept_drafts(target, draft, np.array([[1]], np.int32), u)
    assert a[0] == 0 and t.tolist() == [[0, -1]]
