"""Waits of the prompt attention's kernels: one that runs out is reported, and long regular ones do not run out."""
import math

import pytest
import torch

from prompt_ref import attention

pytestmark = pytest.mark.gpu
D = 128
TIMEOUT = 6


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def long_call(tiles, lk):
    """q, k, v, o of a call whose CTAs, one for each place on the GPU, walk over all lk keys without a split.  Every key
    is zero and every value one, so every weight is alike: o = 1 and lse = log(keys seen), both exactly representable
    sums."""
    Hq, Hkv, lq = (128, 1, 2 * sms()) if tiles == 2 else (2 * sms(), 2 * sms(), 1)
    z = dict(dtype=torch.bfloat16, device="cuda")
    q, k = torch.zeros((lq, Hq, D), **z), torch.zeros((lk, Hkv, D), **z)
    return q, k, torch.ones_like(k), torch.full_like(q, 7.0)


@pytest.fixture
def limit():
    import bit_kv_cache_spc_gb300 as spc
    before = spc.spc_prompt_attn_wait_limit()
    yield spc.spc_prompt_attn_wait_limit
    spc.spc_prompt_attn_wait_limit(before)
    spc.spc_prompt_attn_status()  # cleared


@pytest.mark.parametrize("tiles,lk", [(2, 1 << 19), (1, 1 << 15)])
def test_a_wait_that_runs_out_is_reported(limit, tiles, lk):
    """With a limit of a nanosecond a wait of milliseconds runs out: the workspace's word says so, once, and the next
    call (with the limit of before) is right and reports nothing."""
    import bit_kv_cache_spc_gb300 as spc
    q, k, v, o = long_call(tiles, lk)
    assert spc.spc_prompt_attn_workspace_bytes(q, k, v, o) == 256  # no split
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    before = limit(1)
    spc.spc_prompt_attn(q, k, v, o, ws=ws)
    assert limit(before) == 1
    assert spc.spc_prompt_attn_status(ws) == TIMEOUT
    assert spc.spc_prompt_attn_status(ws) == 0
    assert spc.spc_prompt_attn_status() == TIMEOUT  # the device's word
    o.fill_(7.0)
    spc.spc_prompt_attn(q, k, v, o, ws=ws)
    assert bool((o == 1).all()) and spc.spc_prompt_attn_status(ws) == 0


def test_a_long_walk_over_keys_is_no_wait_that_ran_out(limit):
    """65536 stages of 128 keys: the warps that look after masked places wait for nearly all of the call.  A limit of
    three quarters of its time (with the stages' part, one and a half of it) does not end it."""
    import bit_kv_cache_spc_gb300 as spc
    q, k, v, o = long_call(2, 1 << 23)
    lse = torch.zeros(q.shape[:2], device="cuda")
    spc.spc_prompt_attn(q, k, v, o, lse)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    spc.spc_prompt_attn(q, k, v, o, lse)
    b.record()
    b.synchronize()
    o.fill_(7.0)
    before = limit(int(0.75e6 * a.elapsed_time(b)))
    spc.spc_prompt_attn(q, k, v, o, lse)
    limit(before)
    assert spc.spc_prompt_attn_status() == 0
    assert bool((o == 1).all())
    seen = (1 << 23) - torch.arange(2 * sms() - 1, -1, -1, device="cuda", dtype=torch.float64)
    # log(l) in binary32: within two units of its 15.9
    assert bool(((lse.double() - seen.log()[:, None]).abs() <= 2 * 2.0 ** -20).all())


@pytest.mark.parametrize("split", [False, True])
def test_calls_without_a_workspace_report_to_the_device(limit, split):
    """Also where the call takes its own workspace for the splits: one token, a few heads, a few million keys."""
    import bit_kv_cache_spc_gb300 as spc
    q, k, v, o = long_call(2, 1 << 19)
    if split:
        k, v = (torch.full((1 << 22, 1, D), float(i), dtype=torch.bfloat16, device="cuda") for i in range(2))
        q, o = q[:1, :4].contiguous(), o[:1, :4].contiguous()
        assert spc.spc_prompt_attn_workspace_bytes(q, k, v, o) > 256
    assert spc.spc_prompt_attn_status() == 0
    before = limit(1)
    spc.spc_prompt_attn(q, k, v, o)
    limit(before)
    assert spc.spc_prompt_attn_status() == TIMEOUT
    assert spc.spc_prompt_attn_status() == 0
    spc.spc_prompt_attn(q, k, v, o)
    assert bool((o == 1).all()) and spc.spc_prompt_attn_status() == 0


def test_small_calls_after_one_that_ran_out(limit):
    """Tensor memory and barriers are left as the next calls need them."""
    import bit_kv_cache_spc_gb300 as spc
    q, k, v, o = long_call(2, 1 << 19)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    before = limit(1)
    spc.spc_prompt_attn(q, k, v, o, ws=ws)
    limit(before)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for lq, lk in ((300, 700), (1, 200)):
        q, k, v = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16) for s in ((lq, 8, D), (lk, 2, D), (lk, 2, D)))
        o, lse = torch.zeros_like(q), torch.zeros((lq, 8), device="cuda")
        spc.spc_prompt_attn(q, k, v, o, lse)
        want, z, o_tol, z_tol = attention(q, k, v, 1 / math.sqrt(D))
        assert bool(((o.double() - want).abs() <= o_tol).all()) and bool(((lse.double() - z).abs() <= z_tol).all())
    assert spc.spc_prompt_attn_status(ws) == TIMEOUT
