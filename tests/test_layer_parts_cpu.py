"""The calls around the sequence mixers without a GPU: struct layout, refusals of the
C ABI and of the binding, and the oracle's own pins."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from gated_deltanet_02_gb300 import (glinattn_add_rms_norm, glinattn_kv_append_rope, glinattn_selective_scan_packed,
                                     glinattn_short_conv)
from gated_deltanet_02_gb300 import glinattn as G
from oracle import layer_parts as L
from oracle.selective_scan import selective_scan

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 30                     # addresses far enough apart that no two arrays overlap
INVALID, UNSUPPORTED = 1, 2


def test_struct_layout_matches_header(tmp_path):
    structs = ((G.KvRopeArgs, "glinattn_kv_rope_args"), (G.ShortConvArgs, "glinattn_short_conv_args"),
               (G.ScanPackedArgs, "glinattn_scan_packed_args"), (G.NormArgs, "glinattn_norm_args"))
    src = tmp_path / "layout.c"
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "glinattn.h"', "int main(void){"]
    for ct, name in structs:
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f}));' for f, _ in ct._fields_]
    lines.append('printf("%d\\n", GLINATTN_E8M0);')
    src.write_text("\n".join(lines + ["return 0;}"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for ct, _ in structs:
        want.append(ctypes.sizeof(ct))
        want += [getattr(ct, f).offset for f, _ in ct._fields_]
    assert got == want + [G.E8M0]


def test_packed_bytes_are_the_structs():
    for args, pack in ((G.KvRopeArgs, G._pack_rope), (G.ShortConvArgs, G._pack_conv), (G.ScanPackedArgs, G._pack_scan), (G.NormArgs, G._pack_norm)):
        values = [k + 1.5 if t is ctypes.c_float else (k + 1) * 0x01020304 % (1 << 31) for k, (_, t) in enumerate(args._fields_)]
        got = args.from_buffer_copy(pack(*values))
        assert len(pack(*values)) == ctypes.sizeof(args)
        assert [getattr(got, f) for f, _ in args._fields_] == values


def test_scan_workspace():
    lib = G.library()
    size = lambda **kw: lib.glinattn_selective_scan_packed_workspace_size(ctypes.byref(_scan(**kw)))  # noqa: E731
    long = dict(num_req=1, num_tok=100000, max_q_len=100000, channels=256)
    need = size(**long)
    pieces = 100000 // 512
    assert need >= pieces * 256 * (2 * 16 + 1) * 4 and size(**dict(long, state=12)) == 0
    assert size(**dict(long, max_q_len=1000)) == 0 and size(num_req=0) == 0 and size(**dict(long, num_req=2000)) == 0
    far = dict(x=1 << 40, delta=2 << 40, z=3 << 40, Bm=4 << 40, Cm=5 << 40, y=6 << 40)
    for kw in (dict(), dict(workspace=A), dict(workspace=A, workspace_bytes=need - 1), dict(workspace=A + 8, workspace_bytes=need)):
        assert lib.glinattn_selective_scan_packed(ctypes.byref(_scan(**long, **far, **kw)), None) == INVALID


def _norm(**kw):
    base = dict(in_dtype=G.BF16, residual_dtype=G.BF16, out_dtype=G.BF16, scale_dtype=G.F32, rows=4, width=256, eps=1e-6, x=A,
                residual=2 * A, weight=3 * A, residual_out=4 * A, y=5 * A)
    base.update(kw)
    return G.NormArgs(**base)


E4 = dict(out_dtype=G.E4M3, scale=6 * A)


@pytest.mark.parametrize("kw,code", [
    (dict(in_dtype=G.E4M3), INVALID), (dict(out_dtype=G.E8M0), INVALID), (dict(out_dtype=-1), INVALID), (dict(residual_dtype=G.E4M3), INVALID),
    (dict(rows=-1), INVALID), (dict(width=0), INVALID), (dict(x_stride=-1), INVALID), (dict(x_stride=255), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(residual=None), INVALID), (dict(residual_out=None), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID),
    (dict(x=A + 1), INVALID), (dict(residual=2 * A + 8), INVALID), (dict(y=5 * A + 2), INVALID), (dict(weight=3 * A + 4), INVALID),
    (dict(group=32), INVALID), (dict(scale=6 * A), INVALID), (dict(E4, scale=None), INVALID), (dict(E4, group=16), UNSUPPORTED),
    (dict(E4, group=-32), INVALID), (dict(E4, group=128, width=192), INVALID), (dict(E4, scale_dtype=G.BF16), INVALID),
    (dict(E4, scale=6 * A + 4), INVALID),
    # outputs on inputs other than exactly their own place, and on each other
    (dict(y=A + 16), INVALID), (dict(y=A, in_dtype=G.F32), INVALID), (dict(y=A, x_stride=264), INVALID), (dict(y=2 * A), INVALID),
    (dict(y=3 * A), INVALID), (dict(residual_out=2 * A + 512), INVALID), (dict(residual_out=A, residual_dtype=G.F32), INVALID),
    (dict(residual_out=5 * A), INVALID), (dict(E4, y=A), INVALID), (dict(E4, scale=A), INVALID), (dict(E4, scale=5 * A + 512), INVALID),
])
def test_norm_refusals(kw, code):
    assert G.library().glinattn_add_rms_norm(ctypes.byref(_norm(**kw)), None) == code


def _conv(**kw):
    base = dict(in_dtype=G.BF16, num_req=2, num_tok=6, channels=64, width=4, activation=1, pool_slots=8, update_state=1, x=A, w=2 * A,
                bias=3 * A, conv_pool=4 * A, slot_ids=5 * A, q_start=6 * A, y=7 * A)
    base.update(kw)
    return G.ShortConvArgs(**base)


PACKED = [
    (dict(in_dtype=G.E4M3), INVALID), (dict(num_req=-1), INVALID), (dict(num_req=65536), UNSUPPORTED), (dict(num_tok=-1), INVALID),
    (dict(num_tok=(1 << 30) + 1), UNSUPPORTED), (dict(channels=0), INVALID), (dict(channels=(1 << 20) + 1), UNSUPPORTED), (dict(slot_ids=None), INVALID), (dict(pool_slots=0), INVALID),
    (dict(q_start=None), INVALID), (dict(slot_ids=5 * A + 2), INVALID), (dict(q_start=6 * A + 1), INVALID), (dict(resume=9 * A + 2), INVALID),
    (dict(count=9 * A + 2), INVALID), (dict(x=None), INVALID), (dict(x=A + 1), INVALID), (dict(x_stride=63), INVALID),
    (dict(x_stride=-64), INVALID), (dict(y=7 * A + 8), INVALID), (dict(y=A), INVALID), (dict(y=4 * A), INVALID),
    (dict(y=None, update_state=0), INVALID),
]


@pytest.mark.parametrize("kw,code", PACKED + [
    (dict(width=1), UNSUPPORTED), (dict(width=5), UNSUPPORTED), (dict(activation=2), INVALID), (dict(w=None), INVALID),
    (dict(w=2 * A + 4), INVALID), (dict(bias=3 * A + 4), INVALID), (dict(conv_pool=None), INVALID), (dict(conv_pool=4 * A + 2), INVALID),
    (dict(conv_pool=A + 64), INVALID), (dict(y=None, conv_pool=None, slot_ids=None), INVALID),
])
def test_conv_refusals(kw, code):
    assert G.library().glinattn_short_conv(ctypes.byref(_conv(**kw)), None) == code


def _scan(**kw):
    base = dict(in_dtype=G.BF16, out_dtype=G.BF16, num_req=2, num_tok=6, channels=64, state=16, pool_slots=8, update_state=1, max_q_len=6,
                x=A, delta=2 * A, z=3 * A, Bm=8 * A, Cm=9 * A, A=10 * A, skip=11 * A, delta_bias=12 * A, state_pool=4 * A, slot_ids=5 * A,
                q_start=6 * A, y=7 * A)
    base.update(kw)
    return G.ScanPackedArgs(**base)


@pytest.mark.parametrize("kw,code", PACKED + [
    (dict(out_dtype=G.E4M3), INVALID), (dict(state=12), UNSUPPORTED), (dict(state=64), UNSUPPORTED), (dict(state=0), INVALID),
    (dict(max_q_len=-1), INVALID), (dict(delta=None), INVALID), (dict(Bm=None), INVALID), (dict(Cm=None), INVALID), (dict(A=None), INVALID),
    (dict(A=10 * A + 4), INVALID), (dict(skip=11 * A + 4), INVALID), (dict(delta_bias=12 * A + 4), INVALID), (dict(state_pool=None), INVALID),
    (dict(state_pool=4 * A + 8), INVALID), (dict(z=3 * A + 1), INVALID), (dict(delta_stride=8), INVALID), (dict(b_stride=15), INVALID),
    (dict(c_stride=-16), INVALID), (dict(z_stride=63), INVALID), (dict(y=9 * A), INVALID), (dict(state_pool=2 * A), INVALID),
])
def test_scan_refusals(kw, code):
    assert G.library().glinattn_selective_scan_packed(ctypes.byref(_scan(**kw)), None) == code


def _rope(**kw):
    base = dict(cache_dtype=G.BF16, num_req=2, num_tok=4, heads=4, kv_heads=2, head_dim=128, page_size=16, num_pages=8, max_pages=4,
                rotary_dim=128, rope_scale=1.0, q=A, k=2 * A, v=3 * A, inv_freq=4 * A, q_out=5 * A, k_cache=6 * A, v_cache=7 * A,
                page_table=8 * A, kv_len=9 * A, q_start=10 * A)
    base.update(kw)
    return G.KvRopeArgs(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(cache_dtype=G.F32), INVALID), (dict(num_req=65537), INVALID), (dict(num_tok=-1), INVALID), (dict(kv_heads=0), INVALID),
    (dict(heads=-1), INVALID), (dict(heads=70000), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
    (dict(rotary_dim=0), INVALID), (dict(rotary_dim=144), INVALID), (dict(rotary_dim=40), UNSUPPORTED), (dict(rope_scale=0.0), INVALID),
    (dict(rope_scale=float("nan")), INVALID), (dict(rope_scale=float("inf")), INVALID), (dict(q=None), INVALID), (dict(q_out=None), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(inv_freq=None), INVALID), (dict(inv_freq=4 * A + 2), INVALID),
    (dict(q=A + 8), INVALID), (dict(k=2 * A + 8), INVALID), (dict(q_stride=504), INVALID), (dict(k_stride=260), INVALID),
    (dict(v_stride=-256), INVALID), (dict(cache_dtype=G.E4M3), INVALID), (dict(kv_len=None), INVALID), (dict(q_start=None), INVALID),
    (dict(q_out=A + 256), INVALID),                                     # q_out on part of q
    (dict(q_out=A, q_stride=1024), INVALID),                            # in place with another distance of rows
    (dict(q_out=2 * A - 256), INVALID),                                 # into k
    (dict(q_out=A, k=A + 512, q_stride=1024, q_out_stride=1024, k_stride=1024), INVALID),
])
def test_rope_refusals(kw, code):
    assert G.library().glinattn_kv_append_rope(ctypes.byref(_rope(**kw)), None) == code


def test_empty_calls_launch_nothing():
    lib = G.library()
    for name, args in (("glinattn_add_rms_norm", _norm(rows=0, x=None)), ("glinattn_short_conv", _conv(num_tok=0, x=None)),
                       ("glinattn_short_conv", _conv(num_req=0, x=None)), ("glinattn_selective_scan_packed", _scan(num_tok=0, x=None)),
                       ("glinattn_kv_append_rope", _rope(num_tok=0, k=None))):
        assert getattr(lib, name)(ctypes.byref(args), None) == 0
        assert getattr(lib, name)(None, None) == INVALID


def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def _i(*s):
    return torch.zeros(*s, dtype=torch.int32)


def test_binding_checks_of_the_norm():
    x = _bf(4, 96)
    for bad, kind in ((dict(weight=torch.zeros(95)), ValueError), (dict(weight=_bf(96)), TypeError), (dict(residual=_bf(4, 95)), ValueError),
                      (dict(residual_out=_bf(4, 96)), ValueError), (dict(residual=_bf(4, 96).half()), TypeError),
                      (dict(out_dtype=torch.float16), TypeError), (dict(group=32), ValueError), (dict(scale=torch.zeros(4, 1)), ValueError),
                      (dict(out_dtype=torch.float8_e4m3fn, group=64), ValueError), (dict(out_dtype=torch.float8_e4m3fn, group=48), ValueError),
                      (dict(out_dtype=torch.float8_e4m3fn, scale_dtype=torch.bfloat16), TypeError),
                      (dict(out_dtype=torch.float8_e4m3fn, scale=torch.zeros(4, 2)), ValueError),
                      (dict(y=_bf(4, 96), out_dtype=torch.float32), TypeError), (dict(), ValueError)):     # the last: not on a GPU
        with pytest.raises(kind):
            glinattn_add_rms_norm(x, **bad)
    with pytest.raises(ValueError):
        glinattn_add_rms_norm(_bf(96, 4).T)
    with pytest.raises(ValueError):
        glinattn_add_rms_norm(_bf(1, 96).expand(4, 96))


def test_binding_checks_of_the_packed_calls():
    x, w, pool, slots, qs = _bf(6, 32), torch.zeros(32, 4), _bf(5, 3, 32), _i(2), _i(3)
    for args, kw, kind in (((x, w[:, :3].contiguous(), None, pool, slots, qs), {}, ValueError), ((x, w, None, pool, None, qs), {}, ValueError),
                           ((x, w, None, pool, _i(3), qs), {}, ValueError), ((x, w, None, pool.float(), slots, qs), {}, TypeError),
                           ((x, w, torch.zeros(31), pool, slots, qs), {}, ValueError), ((x, w.double(), None, pool, slots, qs), {}, TypeError),
                           ((x, w, None, pool, slots, qs), dict(resume=_i(3)), ValueError), ((x, w, None, pool, slots, qs), dict(y=_bf(6, 31)), ValueError),
                           ((x, w, None, pool, slots, qs), dict(y=_bf(6, 32), outputs=False), ValueError),
                           ((x, w, None, pool, slots), {}, ValueError), ((x.half(), w, None, pool, slots, qs), {}, TypeError),
                           ((x, w, None, pool, slots, qs), {}, ValueError)):                               # not on a GPU
        with pytest.raises(kind):
            glinattn_short_conv(*args, **kw)
    B, A_, sp = _bf(6, 16), torch.zeros(32, 16), torch.zeros(5, 32, 16)
    for args, kw, kind in (((x, x, B, _bf(6, 8), A_, sp, slots, qs), {}, ValueError), ((x, x.float(), B, B, A_, sp, slots, qs), {}, TypeError),
                           ((x, x, B, B, A_, sp.half(), slots, qs), {}, TypeError), ((x, x, B, B, A_, sp, slots, qs), dict(skip=torch.zeros(16)), ValueError),
                           ((x, x, B, B, A_, sp, slots, qs), dict(max_q_len=1 << 31), ValueError), ((x, x, B, B, A_, sp, slots, qs), dict(max_q_len=-1), ValueError),
                           ((x, x, B, B, A_, sp, slots, qs), dict(z=_bf(6, 16)), ValueError), ((x, x, B, B, A_, sp, slots, qs), dict(out_dtype=torch.float16), TypeError),
                           ((x, x, B, B, A_, sp, slots, qs), dict(dev_status=torch.zeros(1)), ValueError), ((x, x, B, B, A_, sp, slots, qs), {}, ValueError)):
        with pytest.raises(kind):
            glinattn_selective_scan_packed(*args, **kw)


def test_binding_checks_of_the_rotation():
    q, k, f, cache = _bf(3, 4, 64), _bf(3, 2, 64), torch.zeros(32), _bf(4, 2, 16, 64)
    rest = (cache, cache, _i(2, 3), _i(2), _i(3))
    for args, kw, kind in (((q, k, k, f.double(), *rest), {}, TypeError), ((q, k, k, torch.zeros(2, 16), *rest), {}, ValueError),
                           ((q, k[:2], k, f, *rest), {}, ValueError), ((q[..., :32], k, k, f, *rest), {}, ValueError),
                           ((q.transpose(0, 1).contiguous().transpose(0, 1), k, k, f, *rest), {}, ValueError), ((None, k, k, f, *rest), dict(q_out=q), ValueError),
                           ((q, k.float(), k, f, *rest), {}, TypeError), ((q, k, k, f, *rest), dict(k_scale=torch.zeros(4, 2, 16, dtype=torch.uint8)), ValueError),
                           ((q, k, k, f, *rest), {}, ValueError)):
        with pytest.raises(kind):
            glinattn_kv_append_rope(*args, **kw)


def test_oracle_norm_and_rotation_pins():
    y, h = L.add_rms_norm(np.array([[3.0, 4.0]]), np.array([[0.0, 0.0]]), np.array([1.0, 2.0]), 0.0)
    assert np.allclose(y, [[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]]) and np.array_equal(h, [[3.0, 4.0]])
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    y, _ = L.rotate(x, [1], [math.pi / 2, math.pi])
    assert np.allclose(y, [[[-3.0, -2.0, 1.0, -4.0, 5.0]]])
    y, _ = L.rotate(x, [1], [math.pi / 2, math.pi], interleaved=True, scale=2.0)
    assert np.allclose(y, [[[-4.0, 2.0, -6.0, -8.0, 5.0]]])
    # a whole number of turns far out, against exact integer arithmetic: 2^40 * f for f = 2 pi / 3 rounded to fp32
    f = float(np.float32(2 * math.pi / 3))
    y, _ = L.rotate(np.array([[[1.0, 0.0]]]), [1 << 28], [f])
    turn = (1 << 28) * f / (2 * math.pi)
    assert abs(y[0, 0, 0] - math.cos(2 * math.pi * (turn - round(turn)))) < 1e-6


def test_oracle_conv_pins():
    x = np.arange(1.0, 7.0)[:, None]
    w = np.array([[1.0, 10.0, 100.0]])
    pool = np.array([[[7.0], [8.0]], [[0.5], [0.25]]])
    y, size, new = L.short_conv(x, w, np.array([0.5]), pool, [1, 0], np.array([0, 4, 6]), resume=[1, 0], act=False)
    assert np.allclose(y[:, 0], [0.5 + 2.5 + 100.5, 0.25 + 10 + 200.5, 321.5, 432.5, 500.5, 650.5])
    assert np.array_equal(new, [[[5.0], [6.0]], [[3.0], [4.0]]]) and np.allclose(size, y)
    y, _, new = L.short_conv(x, w, None, pool, [1, 0], np.array([0, 4, 6]), count=[1, 0], act=False)
    assert np.isnan(y[1:]).all() and np.array_equal(new, [[[7.0], [8.0]], [[0.25], [1.0]]])


def test_oracle_scan_is_the_plain_scan():
    g = np.random.default_rng(1)
    D, N, lens = 5, 8, [3, 0, 4]
    n = sum(lens)
    x, d, B, C, A_ = g.normal(size=(n, D)), g.normal(size=(n, D)), g.normal(size=(n, N)), g.normal(size=(n, N)), -np.exp(g.normal(size=(D, N)))
    pool = g.normal(size=(4, D, N))
    y, _, new, _, _ = L.scan_packed(x, d, B, C, A_, pool, [2, 0, 1], np.array([0, 3, 3, 7]))
    for (a, b), s in (((0, 3), 2), ((3, 7), 1)):
        yr, hr = selective_scan(x[None, a:b], d[None, a:b], B[None, a:b], C[None, a:b], A_, pool[s][None])
        assert np.allclose(y[a:b], yr[0]) and np.allclose(new[s], hr[0])
    assert np.array_equal(new[[0, 3]], pool[[0, 3]])
    z, D_, b = g.normal(size=(n, D)), g.normal(size=D), g.normal(size=D)
    y2, *_ = L.scan_packed(x, d - b, B, C, A_, pool, [2, 0, 1], np.array([0, 3, 3, 7]), z=z, skip=D_, bias=b)
    assert np.allclose(y2, (y + D_ * x) * z / (1 + np.exp(-z)))
