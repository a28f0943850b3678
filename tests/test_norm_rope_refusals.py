"""Refusals of spc_norm_rope and spc_rope_axes: every bad call comes back before anything reaches the GPU."""
import ctypes as C
import math

import pytest
import torch

import bit_kv_cache_spc_gb300 as spc
from bit_kv_cache_spc_gb300 import _lib, spc_layout, spc_norm_rope_dims, spc_rope_dims

INVALID, UNSUPPORTED = 1, 2


def dense(h, T=8):
    return spc_layout(T * h * 128, h * 128, 128)


def call(fn="spc_norm_rope", axes=1, eps=1e-6, axis=(), pos=16, turns=16, wq=64, wk=64, q=1 << 16, k=1 << 20, v=None,
         q_out=-1, k_out=-1, v_out=None, **over):
    """B = 2, T = 8, four query and two KV heads."""
    r = spc_rope_dims(2, 8, 4, 2, 128, 128, 0, 1.0, dense(4), dense(2), dense(2), dense(4), dense(2), dense(2))
    for n, x in over.items():
        setattr(r, n, x)
    d = spc_norm_rope_dims(r, axes, eps, (C.c_uint8 * 64)(*axis))
    return getattr(_lib, fn)(C.byref(d), pos, turns, wq, wk, q, k, v, q if q_out == -1 else q_out, k if k_out == -1 else k_out,
                             v_out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(axes=0), INVALID), (dict(axes=5), INVALID), (dict(axes=2, axis=[0] * 63 + [2]), INVALID), (dict(axis=[0, 1]), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(wq=66), INVALID), (dict(wk=65), INVALID), (dict(q=None, Hq=0, q_out=None), INVALID),
    (dict(k=None, Hkv=0, k_out=None), INVALID),  # a weight without its rows
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(D=64), UNSUPPORTED), (dict(rot=24), UNSUPPORTED),
    (dict(interleaved=2), INVALID), (dict(mscale=math.nan), INVALID), (dict(pos=None), INVALID), (dict(turns=20), INVALID),
    (dict(q=(1 << 16) + 8), INVALID), (dict(v=1 << 24), INVALID), (dict(q_out=(1 << 16) + 256), INVALID),
    (dict(q_out=1 << 30, k_out=1 << 30), INVALID)])
def test_refused(kw, status):
    assert call(**kw) == status and call("spc_norm_rope_check", **kw) == status


@pytest.mark.parametrize("kw", [
    dict(), dict(wq=None), dict(wk=None, wq=None, eps=0.0), dict(axes=4, axis=[i % 4 for i in range(64)]),
    dict(rot=64, axis=[0] * 32 + [9] * 32),  # what stands behind the pairs is not read
    dict(q=None, Hq=0, q_out=None, wq=None), dict(v=1 << 24, v_out=1 << 26)])
def test_taken(kw):
    assert call("spc_norm_rope_check", **kw) == 0


def test_of_nothing_is_nothing():
    assert call(T=0) == 0


def test_axes_of_sections():
    assert spc.spc_rope_axes([64]) == [0] * 64
    assert spc.spc_rope_axes([16, 24, 24]) == [0] * 16 + [1] * 24 + [2] * 24
    assert spc.spc_rope_axes([0, 5, 0, 3], 16) == [1] * 5 + [3] * 3
    got = spc.spc_rope_axes([24, 20, 20], 128, "turns")
    assert got[:6] == [0, 1, 2, 0, 1, 2] and got[60:] == [0] * 4 and [got.count(a) for a in range(3)] == [24, 20, 20]
    assert spc.spc_rope_axes([5, 3], 16, "turns") == [0, 1, 0, 1, 0, 1, 0, 0]


@pytest.mark.parametrize("sections,rot,order,status", [
    ([], 128, "sections", INVALID), ([64, 0, 0, 0, 0], 128, "sections", INVALID), ([32], 128, "sections", INVALID),
    ([65, -1], 128, "sections", INVALID), ([30, 40], 128, "sections", INVALID), ([12], 24, "sections", UNSUPPORTED),
    ([3, 5], 16, "turns", INVALID), ([0, 0], 0, "sections", UNSUPPORTED)])
def test_axes_refused(sections, rot, order, status):
    with pytest.raises(spc.SpcError) as e:
        spc.spc_rope_axes(sections, rot, order)
    assert e.value.status == status
    assert _lib.spc_rope_axes(None, 1, 0, 128, (C.c_uint8 * 64)()) == INVALID
    assert _lib.spc_rope_axes((C.c_int32 * 1)(64), 1, 2, 128, (C.c_uint8 * 64)()) == INVALID
    assert _lib.spc_rope_axes((C.c_int32 * 1)(64), 1, 0, 128, None) == INVALID


def test_tensors_of_the_host_are_refused():
    x = torch.zeros((1, 4, 2, 128), dtype=torch.bfloat16)
    pos = torch.zeros((1, 4), dtype=torch.int32)
    with pytest.raises(ValueError):
        spc.spc_norm_rope(x, None, pos, torch.zeros(64, dtype=torch.int64))
    with pytest.raises(ValueError):
        spc.spc_norm_rope(None, None, pos, pos)
    with pytest.raises(ValueError):
        spc.spc_rope_axes([64], order="rows")
