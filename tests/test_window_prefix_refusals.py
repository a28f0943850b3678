"""Refusals of spc_window_attn and spc_prefix_attn: every bad call comes back before anything reaches the GPU."""
import ctypes as C
import math

import pytest
import torch

import bit_kv_cache_spc_gb300 as spc
from bit_kv_cache_spc_gb300 import _lib, spc_layout, spc_prefix, spc_prompt_dims

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5


def lay(b, t, h):
    return spc_layout(b, t, h)


def dims(**over):
    d = spc_prompt_dims(2, 8, 2, 128, 64, 96, 64, 96, 0.1, lay(64 * 1024, 1024, 128), lay(96 * 256, 256, 128),
                        lay(96 * 256, 256, 128), lay(64 * 1024, 1024, 128))
    for n, x in over.items():
        setattr(d, n, x)
    return d


def window_args(window=10, sinks=2, d=None, **over):
    a = dict(q=1 << 30, k=1 << 31, v=1 << 32, q_begin=None, q_len=None, k_begin=None, k_len=None, o=1 << 33, lse=None,
             ws=4096, ws_bytes=1 << 20)
    a.update(over)
    return (C.byref(dims() if d is None else d), window, sinks, *a.values(), None)


def prefix_args(d=None, tokens=100, pl=None, vl=None, p=0, **over):
    p = spc_prefix(tokens, lay(0, 256, 128) if pl is None else pl, lay(0, 256, 128) if vl is None else vl) if p == 0 else p
    a = dict(q=1 << 30, pk=1 << 35, pv=1 << 36, p_len=None, k=1 << 31, v=1 << 32, q_begin=None, q_len=None, k_begin=None,
             k_len=None, o=1 << 33, lse=None, ws=4096, ws_bytes=1 << 26)
    a.update(over)
    return (C.byref(dims() if d is None else d), None if p is None else C.byref(p), *a.values(), None)


CALLS = {"spc_window_attn": window_args, "spc_prefix_attn": prefix_args}


@pytest.mark.parametrize("fn", CALLS)
@pytest.mark.parametrize("over,status", [
    (dict(S=0), INVALID), (dict(Hkv=3), INVALID), (dict(D=64), UNSUPPORTED), (dict(Hq=258, Hkv=2), UNSUPPORTED),
    (dict(q_max=65), INVALID), (dict(k_max=97), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=0.0), INVALID),
    (dict(o=lay(0, 1024, 128)), INVALID), (dict(k=lay(96 * 256, 0, 128)), INVALID), (dict(q_tokens=1 << 30, q_max=4), UNSUPPORTED),
    (dict(q=lay(0, 1024, 128), o=lay(0, 1024, 128)), INVALID)])
def test_shapes(fn, over, status):
    args = CALLS[fn](d=dims(**over))
    assert getattr(_lib, fn)(*args) == status and getattr(_lib, fn + "_check")(*args) == status


@pytest.mark.parametrize("fn", CALLS)
@pytest.mark.parametrize("over,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(o=None), INVALID), (dict(q=(1 << 30) + 8), INVALID),
    (dict(ws=4104), INVALID), (dict(ws_bytes=255), WORKSPACE), (dict(o=1 << 31), INVALID), (dict(lse=(1 << 30) + 64), INVALID),
    (dict(lse=(1 << 34) + 2), INVALID), (dict(q_len=(1 << 34) + 1), INVALID), (dict(ws=1 << 33), INVALID)])
def test_arguments(fn, over, status):
    args = CALLS[fn](**over)
    assert getattr(_lib, fn)(*args) == status and getattr(_lib, fn + "_check")(*args) == status


@pytest.mark.parametrize("window,sinks", [(0, 0), (-1, 4), (5, -1)])
def test_windows(window, sinks):
    assert _lib.spc_window_attn(*window_args(window, sinks)) == INVALID
    assert _lib.spc_window_attn_workspace_bytes(C.byref(dims()), window, sinks) == 0


@pytest.mark.parametrize("over,status", [
    (dict(p=None), INVALID), (dict(tokens=-1), INVALID), (dict(tokens=1 << 30), UNSUPPORTED), (dict(pk=None), INVALID),
    (dict(pv=None), INVALID), (dict(pk=(1 << 35) + 8), INVALID), (dict(pv=(1 << 36) + 2), INVALID), (dict(p_len=(1 << 34) + 2), INVALID),
    (dict(pl=lay(0, 128, 128)), INVALID), (dict(vl=lay(0, 256, 64)), INVALID), (dict(vl=lay(0, 0, 128)), INVALID),
    (dict(o=1 << 35), INVALID), (dict(o=(1 << 36) + 2 * 100 * 256 - 16), INVALID), (dict(lse=(1 << 35) + 64), INVALID),
    (dict(ws=(1 << 36) + 16), INVALID)])
def test_prefixes(over, status):
    args = prefix_args(**over)
    assert _lib.spc_prefix_attn(*args) == status and _lib.spc_prefix_attn_check(*args) == status


@pytest.mark.parametrize("fn", CALLS)
def test_taken(fn):
    assert getattr(_lib, fn + "_check")(*CALLS[fn]()) == 0
    assert getattr(_lib, fn)(*CALLS[fn](d=dims(q_max=0))) == 0  # no queries: nothing to do


def test_prefixes_taken():
    assert _lib.spc_prefix_attn_check(*prefix_args(tokens=0, pk=None, pv=None)) == 0
    assert _lib.spc_prefix_attn_check(*prefix_args(d=dims(k_max=0), k=None, v=None)) == 0
    assert _lib.spc_prefix_attn_check(*prefix_args(pk=1 << 31, pv=1 << 32)) == 0  # the prefix in the sequences' own buffers


def test_workspaces():
    """Those of the plain attention where it is called; otherwise by what is seen."""
    kl = lay(8192 * 256, 256, 128)
    one = dims(q_max=1, k_tokens=8192, k_max=8192, k=kl, v=kl)
    plain = _lib.spc_prompt_attn_workspace_bytes(C.byref(one))
    assert plain > 256 and _lib.spc_window_attn_workspace_bytes(C.byref(one), 8192, 3) == plain
    assert _lib.spc_window_attn_workspace_bytes(C.byref(one), 4096, 3) == 256  # single tokens join on the chip
    two = dims(q_max=2, k_tokens=8192, k_max=8192, k=kl, v=kl)
    assert _lib.spc_window_attn_workspace_bytes(C.byref(two), 4096, 3) > 256
    assert _lib.spc_window_attn_workspace_bytes(C.byref(two), 64, 0) == 256  # two blocks of keys: no split
    p = spc_prefix(0, lay(0, 256, 128), lay(0, 256, 128))
    assert _lib.spc_prefix_attn_workspace_bytes(C.byref(one), C.byref(p)) == plain
    assert _lib.spc_prefix_attn_workspace_bytes(C.byref(one), None) == 0
    small = dims(q_max=2)
    p.tokens = 30000
    need = _lib.spc_prefix_attn_workspace_bytes(C.byref(small), C.byref(p))
    assert need > 256 and _lib.spc_prefix_attn(*prefix_args(d=small, tokens=30000, ws=None, ws_bytes=0)) == INVALID
    assert _lib.spc_prefix_attn(*prefix_args(d=small, tokens=30000, ws_bytes=need - 1)) == WORKSPACE


def test_tensors_of_the_host_are_refused():
    x = torch.zeros((1, 4, 2, 128), dtype=torch.bfloat16)
    for call in (lambda: spc.spc_window_attn(x, x, x, x.clone(), 4), lambda: spc.spc_window_attn_workspace_bytes(x, x, x, x, 4),
                 lambda: spc.spc_prefix_attn(x, x[0], x[0], x, x, x.clone()),
                 lambda: spc.spc_prefix_attn_workspace_bytes(x, x[0], x[0], x, x, x)):
        with pytest.raises(ValueError):
            call()
