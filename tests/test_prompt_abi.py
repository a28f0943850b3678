"""Refusals of the prompt path's entry points: every bad call comes back before anything reaches the GPU."""
import ctypes as C
import math

import pytest
import torch

import bit_kv_cache_spc_gb300 as spc
from bit_kv_cache_spc_gb300 import _lib, spc_layout, spc_prompt_dims, spc_rope_dims, spc_rope_scaling

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5


def lay(b, t, h):
    return spc_layout(b, t, h)


# ------------------------------------------------------------------------------------------------ rotary positions
def test_frequencies_of_every_rule():
    turns, m = spc.spc_rope_frequencies(128, 10000.0)
    assert m == 1.0
    for i, t in enumerate(turns.tolist()):
        f = 10000.0 ** (-2 * i / 128)
        assert abs(t - f / (2 * math.pi) * 2 ** 64) <= 2 ** 64 * f / (2 * math.pi) * 2 ** -50 + 1
    plain = turns.double()
    lin, _ = spc.spc_rope_frequencies(128, 10000.0, "linear", 4.0)
    assert float((lin.double() / plain - 0.25).abs().max()) < 1e-10
    bands, m = spc.spc_rope_frequencies(128, 10000.0, "bands", 8.0, 1.0, 4.0, 8192.0)
    r = bands.double() / plain
    n = plain * 2.0 ** -64 * 8192.0
    assert m == 1.0 and float((r[n >= 4] - 1).abs().max()) < 1e-9 and float((r[n <= 1] - 0.125).abs().max()) < 1e-9
    mid = (n > 1) & (n < 4)
    mix = (n[mid] - 1) / 3
    assert bool(mid.any()) and float((r[mid] - (mix + (1 - mix) / 8)).abs().max()) < 1e-9
    ramp, m = spc.spc_rope_frequencies(128, 10000.0, "ramp", 16.0, 1.0, 32.0, 4096.0)
    r = ramp.double() / plain
    assert abs(m - (0.1 * math.log(16.0) + 1)) < 1e-6
    # pairs with 32 and with 1 turn in 4096 positions: 64 ln(4096 / (2 pi n)) / ln 10000 = 20.9 and 45.0 (rounded out)
    assert float((r[:21] - 1).abs().max()) < 1e-9 and float((r[47:] - 1 / 16).abs().max()) < 1e-9
    assert bool((r.diff()[20:44] < 0).all())


@pytest.mark.parametrize("rot,kw,status", [
    (0, {}, UNSUPPORTED), (8, {}, UNSUPPORTED), (144, {}, UNSUPPORTED), (40, {}, UNSUPPORTED), (-16, {}, UNSUPPORTED),
    (64, dict(theta=1.0), INVALID), (64, dict(theta=math.nan), INVALID), (64, dict(theta=math.inf), INVALID),
    (64, dict(kind="linear", factor=0.5), INVALID), (64, dict(kind="bands", factor=8.0, low=4.0, high=4.0), INVALID),
    (64, dict(kind="ramp", factor=8.0, low=0.0), INVALID), (64, dict(kind="ramp", factor=8.0, context=0.0), INVALID),
    (64, dict(kind="bands", factor=math.inf), INVALID)])
def test_frequencies_refuse(rot, kw, status):
    with pytest.raises(spc.SpcError) as e:
        spc.spc_rope_frequencies(rot, **kw)
    assert e.value.status == status


def test_frequencies_refuse_an_unknown_rule():
    m = C.c_float()
    buf = (C.c_uint64 * 64)()
    s = spc_rope_scaling(9, 10000.0, 1.0, 1.0, 4.0, 8192.0)
    assert _lib.spc_rope_frequencies(C.byref(s), 128, buf, C.byref(m)) == INVALID
    assert _lib.spc_rope_frequencies(None, 128, buf, C.byref(m)) == INVALID


def dense(h, T=8):
    return lay(T * h * 128, h * 128, 128)


def rope_call(q=1 << 16, k=1 << 20, v=None, q_out=-1, k_out=-1, v_out=None, pos=16, turns=16, ql=None, **over):
    """B = 2, T = 8, four query and two KV heads; q takes 16 KB, k and v 8 KB."""
    d = spc_rope_dims(2, 8, 4, 2, 128, 128, 0, 1.0, dense(4), dense(2), dense(2), dense(4), dense(2), dense(2))
    if ql is not None:
        d.q = ql
    for n, x in over.items():
        setattr(d, n, x)
    return _lib.spc_rope(C.byref(d), pos, turns, q, k, v, q if q_out == -1 else q_out, k if k_out == -1 else k_out, v_out,
                         None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(D=64), UNSUPPORTED), (dict(rot=8), UNSUPPORTED),
    (dict(rot=24), UNSUPPORTED), (dict(rot=256), UNSUPPORTED), (dict(interleaved=2), INVALID),
    (dict(mscale=math.inf), INVALID), (dict(mscale=math.nan), INVALID), (dict(pos=None), INVALID),
    (dict(turns=None), INVALID), (dict(turns=20), INVALID), (dict(q=(1 << 16) + 8), INVALID), (dict(Hq=0), INVALID),
    (dict(q_out=None), INVALID), (dict(v=1 << 24), INVALID), (dict(v_out=1 << 24), INVALID), (dict(Hkv=0), INVALID),
    (dict(q_out=(1 << 16) + 256), INVALID), (dict(q_out=(1 << 16) - 16384 + 16), INVALID),  # reach into their own input
    (dict(v=1 << 24, v_out=(1 << 24) + 512), INVALID),
    (dict(q_out=1 << 30, k_out=1 << 30), INVALID), (dict(k_out=1 << 30, v=1 << 24, v_out=(1 << 30) - 128), INVALID),
    (dict(q_out=1 << 30, ql=lay(4096, 512, 64)), INVALID),      # heads overlap
    (dict(q_out=1 << 30, ql=lay(4096, 512, 0)), INVALID),       # a broadcast axis
    (dict(q_out=1 << 30, ql=lay(4096, 384, 128)), INVALID),     # tokens overlap
    (dict(q_out=1 << 30, ql=lay(4096, 516, 128)), INVALID),     # rows off their 16-byte boundaries
    (dict(q_out=1 << 30, ql=lay(-4096, 512, 128)), INVALID), (dict(q_out=1 << 30, ql=lay(4096, 1 << 40, 128)), INVALID)])
def test_rope_refuses(kw, status):
    assert rope_call(**kw) == status


def test_rope_of_nothing_is_nothing():
    assert rope_call(T=0) == 0


# ------------------------------------------------------------------------------------------------ prompt attention
def prompt_dims(**over):
    d = spc_prompt_dims(2, 8, 2, 128, 64, 96, 64, 96, 0.1, lay(64 * 8 * 128, 8 * 128, 128), lay(96 * 256, 256, 128),
                        lay(96 * 256, 256, 128), lay(64 * 8 * 128, 8 * 128, 128))
    for n, x in over.items():
        setattr(d, n, x)
    return d


def prompt_call(d, q=4096, k=4096, v=4096, o=4096, ws=4096, ws_bytes=1 << 40):
    return _lib.spc_prompt_attn(C.byref(d), q, k, v, None, None, None, None, o, None, ws, ws_bytes, None)


@pytest.mark.parametrize("over,status", [
    (dict(S=0), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=3), INVALID), (dict(D=64), UNSUPPORTED),
    (dict(Hq=258, Hkv=2), UNSUPPORTED), (dict(q_max=65), INVALID), (dict(k_max=97), INVALID), (dict(q_max=-1), INVALID),
    (dict(k_tokens=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=math.nan), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=math.inf), INVALID), (dict(o=lay(0, 8 * 128, 128)), INVALID),
    (dict(v=lay(0, 256, 128)), INVALID), (dict(k=lay(96 * 256, 256, 4)), INVALID), (dict(k=lay(96 * 256, 0, 128)), INVALID),
    (dict(k=lay(96 * 128, 256, 128)), INVALID), (dict(o=lay(64 * 8 * 128, 8 * 128, 64)), INVALID),
    (dict(S=1 << 29, q=lay(0, 1024, 128), o=lay(0, 1024, 128), k=lay(0, 256, 128), v=lay(0, 256, 128)), UNSUPPORTED),
    (dict(q_tokens=1 << 30, q_max=4), UNSUPPORTED)])
def test_prompt_attn_refuses_shapes(over, status):
    d = prompt_dims(**over)
    assert prompt_call(d) == status
    assert _lib.spc_prompt_attn_workspace_bytes(C.byref(d)) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(o=None), INVALID),
    (dict(ws=None), INVALID), (dict(q=4104), INVALID), (dict(v=4098), INVALID), (dict(o=4100), INVALID),
    (dict(ws=4104), INVALID), (dict(ws_bytes=16), WORKSPACE)])
def test_prompt_attn_refuses_arguments(kw, status):
    assert prompt_call(prompt_dims(), **kw) == status


def test_prompt_attn_refuses_sequences_on_the_same_rows():
    """Packed queries of two sequences without their first tokens."""
    assert prompt_call(prompt_dims(q=lay(0, 1024, 128), o=lay(0, 1024, 128))) == INVALID


@pytest.mark.parametrize("kw", [dict(), dict(q=1 << 30, k=1 << 31), dict(q=1 << 30, v=1 << 31),
                                dict(k=1 << 30, v=1 << 31, q=4096 + 64 * 8 * 256 * 2 - 256)])
def test_prompt_attn_refuses_an_output_that_reaches_into_an_input(kw):
    assert prompt_call(prompt_dims(), **kw) == INVALID


def test_prompt_attn_of_no_queries_is_nothing():
    assert prompt_call(prompt_dims(q_max=0)) == 0


def test_prompt_attn_without_a_workspace():
    """NULL is for calls that need none, and then with no bytes."""
    kl = lay(8192 * 256, 256, 128)
    split = prompt_dims(q_max=1, k_tokens=8192, k_max=8192, k=kl, v=kl)
    assert prompt_call(split, ws=None, ws_bytes=0) == INVALID
    assert prompt_call(prompt_dims(), ws=None, ws_bytes=256) == INVALID


def test_prompt_attn_workspace_grows_where_the_keys_are_split():
    d = prompt_dims()
    assert _lib.spc_prompt_attn_workspace_bytes(C.byref(d)) == 256  # no key tiles to share out
    kl = lay(8192 * 256, 256, 128)
    one = prompt_dims(q_max=1, k_tokens=8192, k_max=8192, k=kl, v=kl)
    assert _lib.spc_prompt_attn_workspace_bytes(C.byref(one)) > 256


def test_prompt_attn_splits_no_more_sequences_than_a_grid_numbers():
    """Single tokens over one shared, very long row of keys: 65535 sequences may be split, 65536 are not."""
    for S, split in ((65535, True), (65536, False)):
        d = prompt_dims(S=S, Hq=1, Hkv=1, q_tokens=S, q_max=1, k_tokens=1 << 29, k_max=1 << 29, q=lay(0, 128, 128),
                        o=lay(0, 128, 128), k=lay(0, 128, 128), v=lay(0, 128, 128))
        assert (_lib.spc_prompt_attn_workspace_bytes(C.byref(d)) > 256) == split


# ------------------------------------------------------------------------------------------------ the cache
def cache_call(fn, d=None, n=10, k=1 << 32, v=1 << 33, lk=None, lv=None, records=4096, resid=1 << 24, first=0, host=None,
               n_cap=0):
    """B = 2, two KV heads; 100 tokens, 64 of them quantised."""
    d = spc.Dims(2, 4, 2, 100, 16, 1, q_groups_cap=2, resid_cap=48) if d is None else d
    lk, lv = (lay(256 * max(n, 1), 256, 128) if x is None else x for x in (lk, lv))
    if fn == "extend":
        return _lib.spc_extend_kv(C.byref(d), n, k, v, C.byref(lk), C.byref(lv), records, resid, host, n_cap, None)
    return _lib.spc_dequantize_kv(C.byref(d), records, resid, first, n, k, v, C.byref(lk), C.byref(lv), None)


def room():
    return spc.Dims(2, 4, 2, 100, 16, 1, q_groups_cap=8, resid_cap=48)


@pytest.mark.parametrize("fn", ["extend", "read"])
@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(d=room(), records=None, n=60), INVALID),
    (dict(d=room(), resid=None, n=90), INVALID), (dict(k=(1 << 32) + 8), INVALID),
    (dict(d=room(), records=4104, n=60), INVALID), (dict(resid=(1 << 24) + 2), INVALID),
    (dict(lk=lay(2560, 256, 64)), INVALID), (dict(lv=lay(2560, 128, 128)), INVALID), (dict(lv=lay(0, 256, 128)), INVALID),
    (dict(lk=lay(2560, 256, 129)), INVALID), (dict(k=(1 << 24) + 64), INVALID), (dict(v=4096 + 1024), INVALID),
    (dict(d=spc.Dims(2, 4, 2, 100, 16, 3)), INVALID), (dict(d=spc.Dims(2, 16, 2, 100, 16, 1)), UNSUPPORTED)])
def test_cache_calls_refuse(fn, kw, status):
    assert cache_call(fn, **kw) == status


def test_extend_refuses_what_the_cache_cannot_hold():
    assert cache_call("extend", n=40) == INVALID  # records for two groups only
    assert cache_call("extend", d=spc.Dims(2, 4, 2, 100, 16, 1, q_groups_cap=8, resid_cap=38), n=10) == INVALID
    assert cache_call("extend", d=room(), n=10, host=1 << 30, n_cap=109) == INVALID
    assert cache_call("extend", d=room(), n=1 << 30) == INVALID
    assert cache_call("extend", d=room(), n=0) == 0


def test_read_refuses_tokens_that_are_not_there():
    assert cache_call("read", first=-1) == INVALID
    assert cache_call("read", first=91, n=10) == INVALID
    assert cache_call("read", first=2 ** 31 - 1, n=10) == INVALID
    assert cache_call("read", first=100, n=0) == 0


def test_read_refuses_keys_and_values_on_the_same_rows():
    assert cache_call("read", k=1 << 32, v=1 << 32) == INVALID
    assert cache_call("read", k=1 << 32, v=(1 << 32) + 128) == INVALID


# ------------------------------------------------------------------------------------------------ tensors
def test_tensors_of_the_host_are_refused():
    x = torch.zeros((1, 4, 2, 128), dtype=torch.bfloat16)
    pos = torch.zeros((1, 4), dtype=torch.int32)
    d = spc.Dims(1, 2, 2, 100, 16, 1)
    for call in (lambda: spc.spc_rope(x, None, pos, torch.zeros(64, dtype=torch.int64)),
                 lambda: spc.spc_prompt_attn(x, x, x, x.clone()), lambda: spc.spc_extend_kv(d, x, x, None, None),
                 lambda: spc.spc_dequantize_kv(d, None, None, 0, x, x),
                 lambda: spc.spc_prompt_attn(x.float(), x, x, x), lambda: spc.spc_prompt_attn(x.half(), x, x, x), lambda: spc.spc_extend_kv(d, x[0], x[0], None, None),
                 lambda: spc.spc_rope(None, None, pos, pos), lambda: spc.spc_rope(x, None, pos, pos, k_out=x)):
        with pytest.raises(ValueError):
            call()
