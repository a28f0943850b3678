"""More of the prompt path's host side: settings, and calls that are refused before anything reaches the GPU."""
import ctypes as C
import random

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


# ------------------------------------------------------------------------------------------------ outputs on other rows
def fused(heads, T=8, all_heads=8):
    """A view of some heads of a fused projection [2][8][8][128]."""
    return lay(T * all_heads * 128, all_heads * 128, 128)


HEAD, TOKEN = 256, 8 * 256  # bytes, of that projection


@pytest.mark.parametrize("over", [
    dict(q=1 << 20, k=(1 << 20) + 4 * HEAD, v=(1 << 20) + 6 * HEAD, v_out=1 << 30),  # q and k rotated in place, side by side
    dict(q=1 << 20, k=(1 << 20) + 4 * HEAD, v=(1 << 20) + 6 * HEAD, q_out=1 << 30, k_out=1 << 31, v_out=1 << 32),
    dict(q=1 << 20, k=(1 << 30) + 4 * HEAD, q_out=1 << 30, k_out=1 << 31)])  # q's rows go beside k's
def test_rope_takes_views_that_lie_between_one_another(over):
    assert fused_rope(over) == 0


@pytest.mark.parametrize("over", [
    dict(q=1 << 20, k=(1 << 20) + 3 * HEAD),                               # k starts on q's last head
    dict(q=1 << 20, k=(1 << 20) + 6 * HEAD + 128),                         # ends half a row on the next token's q
    dict(q=1 << 20, k=1 << 24, q_out=1 << 30, k_out=(1 << 30) + HEAD),     # one head on
    dict(q=1 << 20, k=1 << 24, q_out=1 << 30, k_out=(1 << 30) + TOKEN),    # one token on
    dict(q=1 << 20, k=1 << 24, q_out=1 << 30, k_out=(1 << 30) - TOKEN),    # one token before
    dict(q=1 << 20, k=1 << 24, q_out=1 << 30, k_out=(1 << 30) + 8 * TOKEN + HEAD),  # one sequence and a head on
    dict(q=1 << 20, k=1 << 24, q_out=1 << 30, k_out=1 << 31, v=1 << 28, v_out=(1 << 30) + 3 * TOKEN + 2 * HEAD),
    dict(q=1 << 20, k=1 << 24, q_out=(1 << 24) + TOKEN, k_out=1 << 31),    # q's rows go where k's are read
    dict(q=1 << 20, k=1 << 24, k_out=(1 << 20) + 2 * TOKEN)])              # k's where q's are turned in place
def test_rope_refuses_outputs_on_other_rows(over):
    assert fused_rope(over) == INVALID


def fused_rope(over):
    d = spc_rope_dims(2, 8, 4, 2, 128, 128, 0, 1.0, *[fused(h) for h in (4, 2, 2, 4, 2, 2)])
    a = dict(v=None, v_out=None, q_out=over["q"], k_out=over["k"])
    a.update(over)
    return _lib.spc_rope_check(*rope_args(d=d, **a))


def test_reading_back_refuses_exactly_the_views_that_share_rows():
    """Keys and values in one buffer of any order of axes, at any distance: refused where one row of each share a byte,
    by all pairs of rows."""
    rng = random.Random(5)
    seen = set()
    for _ in range(3000):
        n = [2, rng.randint(1, 5), 2]  # batch, tokens, heads
        order, strides, span = rng.sample(range(3), 3), [0, 0, 0], 128
        for i in order:
            strides[i] = span + 8 * rng.choice([0, 0, 1, 16, 40])
            span = strides[i] * n[i] if rng.random() < 0.5 else strides[i] * (n[i] - 1) + span
        far = 2 * (sum(s * (m - 1) for s, m in zip(strides, n)) + 256)
        by = rng.choice([16 * rng.randint(-far // 16, far // 16),
                         2 * sum(s * rng.randint(-m, m) for s, m in zip(strides, n)) + rng.choice([0, 0, 240, 256, -256])])
        starts = [2 * (strides[0] * b + strides[1] * t + strides[2] * h) for b in range(n[0]) for t in range(n[1])
                  for h in range(n[2])]
        want = any(abs(x - y - by) < 256 for x in starts for y in starts)
        got = _lib.spc_dequantize_kv_check(*read_args(n=n[1], k=1 << 32, v=(1 << 32) + by, lk=lay(*strides), lv=lay(*strides)))
        assert got == (INVALID if want else 0), (n, strides, by)
        seen.add((want, abs(by) < far))
    assert seen == {(True, True), (False, True), (False, False)}


# ------------------------------------------------------------------------------------------------ lse and workspace
Q_BYTES, K_BYTES, LSE_BYTES = 2 * 64 * 1024 * 2, 2 * 96 * 256 * 2, 2 * 64 * 8 * 4  # of attn_args' call


@pytest.mark.parametrize("over", [
    dict(lse=(1 << 30) + 64), dict(lse=(1 << 30) - LSE_BYTES + 4), dict(lse=(1 << 31) + K_BYTES - 4), dict(lse=1 << 32),
    dict(lse=(1 << 33) + Q_BYTES - 4), dict(ws=1 << 30, ws_bytes=256), dict(ws=(1 << 31) - 240, ws_bytes=256),
    dict(ws=(1 << 32) + K_BYTES - 16, ws_bytes=256), dict(ws=1 << 33, ws_bytes=256),
    dict(lse=1 << 34, ws=(1 << 34) + LSE_BYTES - 16, ws_bytes=256), dict(lse=1 << 34, ws=(1 << 34) - 240, ws_bytes=256)])
def test_attention_refuses_an_lse_or_workspace_on_other_rows(over):
    assert _lib.spc_prompt_attn_check(*attn_args(**over)) == INVALID


@pytest.mark.parametrize("over", [
    dict(lse=(1 << 30) - LSE_BYTES), dict(lse=(1 << 31) + K_BYTES), dict(lse=(1 << 33) + Q_BYTES),
    dict(ws=(1 << 30) - 256, ws_bytes=1 << 20), dict(lse=1 << 34, ws=(1 << 34) + LSE_BYTES, ws_bytes=256)])
def test_attention_takes_an_lse_or_workspace_beside_other_rows(over):
    """Of a workspace, the bytes that the call needs count."""
    assert _lib.spc_prompt_attn_check(*attn_args(**over)) == 0


# ------------------------------------------------------------------------------------------------ arrays off their elements
@pytest.mark.parametrize("name", ["q_begin", "q_len", "k_begin", "k_len", "lse"])
@pytest.mark.parametrize("by", [1, 2, 3])
def test_attention_refuses_arrays_off_their_elements(name, by):
    assert _lib.spc_prompt_attn_check(*attn_args(**{name: (1 << 34) + by})) == INVALID
    assert _lib.spc_prompt_attn_check(*attn_args(**{name: (1 << 34) + 4})) == 0


def test_rope_refuses_positions_off_their_elements():
    assert _lib.spc_rope_check(*rope_args(pos=18)) == INVALID
    assert _lib.spc_rope_check(*rope_args(pos=20)) == 0


def test_the_wait_limit_is_held_to_a_thousand_seconds():
    try:
        spc.spc_prompt_attn_wait_limit(2 ** 63 - 1)
        assert spc.spc_prompt_attn_wait_limit() == 10 ** 12
    finally:
        spc.spc_prompt_attn_wait_limit(2_000_000_000)
