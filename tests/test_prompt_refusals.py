"""More of the prompt path's host side: settings, and calls that are refused before anything reaches the GPU."""
import ctypes as C

import pytest

import bit_kv_cache_spc_gb300 as spc
from bit_kv_cache_spc_gb300 import _lib, spc_layout, spc_prompt_dims, spc_rope_dims

INVALID, WORKSPACE = 1, 5


def lay(b, t, h):
    return spc_layout(b, t, h)


def test_the_wait_limit_is_read_and_set():
    assert spc.spc_prompt_attn_wait_limit() == 2_000_000_000
    try:
        assert spc.spc_prompt_attn_wait_limit(5) == 2_000_000_000
        assert spc.spc_prompt_attn_wait_limit(-1) == 5 and spc.spc_prompt_attn_wait_limit(0) == 5
    finally:
        assert spc.spc_prompt_attn_wait_limit(2_000_000_000) == 5


# ------------------------------------------------------------------------------------------------ checks alone
# Made-up device addresses: a check reads none.
def rope_args(**over):
    d = spc_rope_dims(2, 8, 4, 2, 128, 128, 0, 1.0, *[lay(8 * h * 128, h * 128, 128) for h in (4, 2, 2, 4, 2, 2)])
    a = dict(d=d, pos=16, turns=16, q=1 << 16, k=1 << 20, v=None, q_out=1 << 16, k_out=1 << 20, v_out=None)
    a.update(over)
    return (C.byref(a.pop("d")), *a.values(), None)


def attn_args(q_max=64, **over):
    d = spc_prompt_dims(2, 8, 2, 128, 64, 96, q_max, 96, 0.1, lay(64 * 1024, 1024, 128), lay(96 * 256, 256, 128),
                        lay(96 * 256, 256, 128), lay(64 * 1024, 1024, 128))
    a = dict(q=1 << 30, k=1 << 31, v=1 << 32, q_begin=None, q_len=None, k_begin=None, k_len=None, o=1 << 33, lse=None,
             ws=None, ws_bytes=0)
    a.update(over)
    return (C.byref(d), *a.values(), None)


def cache_args(read=False, n=60, **over):
    d = spc.Dims(2, 4, 2, 100, 16, 1, q_groups_cap=8, resid_cap=48)
    kl = lay(256 * max(n, 1), 256, 128)
    a = dict(k=1 << 32, v=1 << 33, lk=kl, lv=kl, records=4096, resid=1 << 24, first=0, host=None, n_cap=0)
    a.update(over)
    rows, tail = (a["k"], a["v"]), (C.byref(a["lk"]), C.byref(a["lv"]))
    cache = (a["records"], a["resid"])
    if read:
        return (C.byref(d), *cache, a["first"], n, *rows, *tail, None)
    return (C.byref(d), n, *rows, *tail, *cache, a["host"], a["n_cap"], None)


def read_args(**over):
    return cache_args(read=True, **over)


@pytest.mark.parametrize("fn,args,over,status", [
    ("spc_rope", rope_args, {}, 0), ("spc_rope", rope_args, dict(q_out=(1 << 16) + 256), INVALID),
    ("spc_rope", rope_args, dict(pos=None), INVALID),
    ("spc_prompt_attn", attn_args, {}, 0), ("spc_prompt_attn", attn_args, dict(o=1 << 31), INVALID),
    ("spc_prompt_attn", attn_args, dict(q_max=0, q=None), 0), ("spc_prompt_attn", attn_args, dict(ws=4096, ws_bytes=255), WORKSPACE),
    ("spc_extend_kv", cache_args, {}, 0), ("spc_extend_kv", cache_args, dict(n=0, k=None), 0),
    ("spc_extend_kv", cache_args, dict(n=1000), INVALID), ("spc_extend_kv", cache_args, dict(records=None), INVALID),
    ("spc_extend_kv", cache_args, dict(host=4096, n_cap=159), INVALID),
    ("spc_dequantize_kv", read_args, {}, 0), ("spc_dequantize_kv", read_args, dict(n=0, v=None), 0),
    ("spc_dequantize_kv", read_args, dict(first=41), INVALID)], ids=lambda x: str(x) if not callable(x) else "")
def test_checks_alone_say_what_the_call_would(fn, args, over, status):
    assert getattr(_lib, fn + "_check")(*args(**over)) == status
    if status:  # (a call that would be made is not: there is no memory behind it)
        assert getattr(_lib, fn)(*args(**over)) == status
