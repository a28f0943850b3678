"""spc_window_attn over many more pairs of tiles than the GPU has SMs: CTAs take item after item (short windows)."""
import math

import pytest
import torch

from sight_ref import check, i32, rnd, window_sight

pytestmark = pytest.mark.gpu
D = 128


def call(q, k, v, window, sinks, **kw):
    import bit_kv_cache_spc_gb300 as spc
    o = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:-1], 7.0, device="cuda")
    spc.spc_window_attn(q, k, v, o, window, sinks, lse, **kw)
    return o, lse


@pytest.mark.parametrize("lq,lk,Hq,Hkv,window,sinks", [
    (3000, 3000, 32, 32, 200, 0), (3001, 3100, 32, 8, 130, 5), (2999, 2600, 32, 8, 64, 0), (801, 900, 128, 1, 70, 3),
    (1900, 1900, 40, 40, 1, 0), (1153, 1153, 96, 48, 128, 1), (2000, 0, 32, 32, 9, 2), (1000, 2100, 120, 24, 300, 70),
    (3000, 3000, 40, 40, 600, 0), (2300, 2200, 48, 24, 384, 0)])
def test_one_sequence(lq, lk, Hq, Hkv, window, sinks):
    """Also with fewer keys than queries (items without a block), none at all, and a last pair with one tile."""
    q, k, v = rnd(1, lq, Hq, D), rnd(2, lk, Hkv, D), rnd(3, lk, Hkv, D)
    if lk == 0:
        k, v = rnd(2, 1, Hkv, D), rnd(3, 1, Hkv, D)
    n = i32([lk])
    o, lse = call(q, k, v, window, sinks, k_len=n)
    check(o, lse, q, k[:lk], v[:lk], window_sight(lq, lk, window, sinks))
    for _ in range(3):
        again = call(q, k, v, window, sinks, k_len=n)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("Hq,Hkv", [(16, 16), (32, 8), (18, 3)])
@pytest.mark.parametrize("window,sinks", [(100, 0), (190, 70)])
@pytest.mark.parametrize("S", [40, 300])
def test_packed_sequences(Hq, Hkv, window, sinks, S):
    """Sequences of no, one and a few hundred tokens, with and without keys before them: pairs whose second tile is
    missing, items whose rows see nothing, gaps that keep their bytes."""
    import bit_kv_cache_spc_gb300 as spc
    lq = [(0, 1, 127, 129, 300, 64, 521, 33)[(s * 5) % 8] for s in range(S)]
    lk = [max(0, n + (0, 200, -60, 0, 77)[s % 5]) if s % 9 else 0 for s, n in enumerate(lq)]
    qb, kb, T, Tk = [], [], 2, 0
    for n, m in zip(lq, lk):
        qb.append(T)
        kb.append(Tk)
        T, Tk = T + n + 1, Tk + m
    q, k, v = rnd(1, T, Hq, D), rnd(2, Tk, Hkv, D), rnd(3, Tk, Hkv, D)
    at = dict(q_begin=i32(qb), q_len=i32(lq), k_begin=i32(kb), k_len=i32(lk), q_max=max(lq), k_max=max(lk))
    o, lse = call(q, k, v, window, sinks, **at)
    untouched = torch.ones(T, dtype=torch.bool, device="cuda")
    for s, (b, n, c, m) in enumerate(zip(qb, lq, kb, lk)):
        if n and (s < 40 or s >= S - 3):
            check(o[b:b + n], lse[b:b + n], q[b:b + n], k[c:c + m], v[c:c + m], window_sight(n, m, window, sinks))
        untouched[b:b + n] = False
    assert bool((o[untouched] == 7).all()) and bool((lse[untouched] == 7).all())
    assert not bool((lse[~untouched] == 7).any())
    again = call(q, k, v, window, sinks, **at)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    assert spc.spc_prompt_attn_status() == 0


def test_batch_over_head_major_caches():
    """Rows of other strides than whole tiles are stored in, lengths that differ, rows behind them as they were."""
    import bit_kv_cache_spc_gb300 as spc
    S, Hq, Hkv, most, cap = 5, 16, 16, 700, 1000
    lq, lk = [700, 1, 0, 513, 260], [700, 1000, 9, 513, 100]
    qkv = rnd(1, S, most, Hq, 2 * D)
    q = qkv[..., D:]
    k, v = (rnd(i, S, Hkv, cap, D).transpose(1, 2) for i in (2, 3))
    buf = torch.full((S, Hq, most, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    o = buf[..., 8:].transpose(1, 2)
    spc.spc_window_attn(q, k, v, o, 128, 4, q_len=i32(lq), k_len=i32(lk))
    for s, (n, m) in enumerate(zip(lq, lk)):
        if n:
            check(o[s, :n], None, q[s, :n], k[s, :m], v[s, :m], window_sight(n, m, 128, 4))
        assert bool((o[s, n:] == 7).all())
    assert bool((buf[..., :8] == 7).all())


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("sinks", [0, 2])
def test_non_finite_keys_and_values(what, sinks):
    """A poisoned stretch of one head leaves the rows that do not see it bit for bit as they were, in every item that a CTA
    takes before and after; values alone reach the rows that see them with their sign."""
    L, H, window = 2600, 32, 150
    q, k, v = rnd(1, L, H, D), rnd(2, L, H, D), rnd(3, L, H, D)
    o, lse = call(q, k, v, window, sinks)
    kk, vv = k.clone(), v.clone()
    kk[1301:1340, 5], vv[1301:1340, 5] = what, what
    o2, lse2 = call(q, kk, vv, window, sinks)
    clean = torch.ones((L, H), dtype=torch.bool, device="cuda")
    clean[:, 5] = ~window_sight(L, L, window, sinks)[:, 1301:1340].any(1)
    assert int((~clean).sum()) == 39 + window - 1
    assert torch.equal(o[clean], o2[clean]) and torch.equal(lse[clean], lse2[clean])
    vv = v.clone()
    places = [(700 + 37 * i, i) for i in range(H)]  # a key of each head, channel 2 i
    for j, h in places:
        vv[j, h, 2 * h] = what
    o3, lse3 = call(q, k, vv, window, sinks)
    assert torch.equal(lse, lse3)
    hit = torch.zeros_like(o, dtype=torch.bool)
    for j, h in places:
        hit[j:j + window, h, 2 * h] = True
    assert torch.equal(o[~hit], o3[~hit])
    assert bool(torch.isnan(o3[hit]).all() if math.isnan(what) else (o3[hit] == what).all())


@pytest.mark.parametrize("mul", [12.0, 0.0])
def test_growing_and_equal_scores(mul):
    q, k, v = rnd(1, 3000, 32, D, mul=mul), rnd(2, 3000, 16, D), rnd(3, 3000, 16, D)
    o, lse = call(q, k, v, 333, 7)
    check(o, lse, q, k, v, window_sight(3000, 3000, 333, 7))


def test_graphs_and_streams_repeat_the_same_bits():
    """Captured and replayed with other lengths, and two calls at once."""
    import bit_kv_cache_spc_gb300 as spc
    q, k, v = rnd(1, 2000, 32, D), rnd(2, 2000, 16, D), rnd(3, 2000, 16, D)
    n, o, lse = i32([2000]), torch.zeros_like(q), torch.zeros((2000, 32), device="cuda")
    ws = torch.zeros(spc.spc_window_attn_workspace_bytes(q, k, v, o, 128, 1), dtype=torch.uint8, device="cuda")
    spc.spc_window_attn(q, k, v, o, 128, 1, lse, k_len=n, ws=ws)
    want = o.clone(), lse.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        spc.spc_window_attn(q, k, v, o, 128, 1, lse, k_len=n, ws=ws)
    n.fill_(1703)
    g.replay()
    torch.cuda.synchronize()
    check(o, lse, q, k[:1703], v[:1703], window_sight(2000, 1703, 128, 1))
    n.fill_(2000)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    side = [torch.cuda.Stream() for _ in range(2)]
    outs, wss = [torch.zeros_like(o) for _ in side], [torch.zeros_like(ws) for _ in side]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, x, w in zip(side, outs, wss):
            spc.spc_window_attn(q, k, v, x, 128, 1, k_len=n, ws=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[0]) for x in outs)
    assert spc.spc_prompt_attn_status(ws) == 0 and spc.spc_prompt_attn_status() == 0


def test_a_wait_that_runs_out_is_reported():
    """With a limit of a nanosecond: each item's second tile has no rows, and its warps wait for the walk of the first over
    2560 keys.  The next call is right."""
    import bit_kv_cache_spc_gb300 as spc
    lk, S = 2560, 40 * torch.cuda.get_device_properties(0).multi_processor_count
    z = dict(dtype=torch.bfloat16, device="cuda")
    q, k = torch.zeros((S, 128, D), **z), torch.zeros((lk, 1, D), **z)
    v, o, ws = torch.ones_like(k), torch.full_like(q, 7.0), torch.zeros(256, dtype=torch.uint8, device="cuda")
    at = dict(q_begin=torch.arange(S, dtype=torch.int32, device="cuda"), q_len=i32([1] * S), k_begin=i32([0] * S),
              k_len=i32([lk] * S), q_max=2, k_max=lk)
    before = spc.spc_prompt_attn_wait_limit(1)
    try:
        spc.spc_window_attn(q, k, v, o, lk - 1, ws=ws, **at)
        spc.spc_prompt_attn_wait_limit(before)
        assert spc.spc_prompt_attn_status(ws) == 6 and spc.spc_prompt_attn_status(ws) == 0
        assert spc.spc_prompt_attn_status() == 6 and spc.spc_prompt_attn_status() == 0
        spc.spc_window_attn(q, k, v, o, lk - 1, ws=ws, **at)
        assert bool((o == 1).all()) and spc.spc_prompt_attn_status(ws) == 0
    finally:
        spc.spc_prompt_attn_wait_limit(before)
        spc.spc_prompt_attn_status()
