"""The attention with a sliding window and first tokens that stay visible (spc_window_attn) against a plain 64-bit form."""
import math

import pytest
import torch

from sight_ref import check, i32, rnd, window_sight

pytestmark = pytest.mark.gpu
D = 128


def run_one(lq, lk, Hq, Hkv, window, sinks, seed=0, mul=1.0, **kw):
    import bit_kv_cache_spc_gb300 as spc
    q, k, v = rnd(seed, lq, Hq, D, mul=mul), rnd(seed + 1, lk, Hkv, D), rnd(seed + 2, lk, Hkv, D)
    o = torch.full((lq, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((lq, Hq), 7.0, device="cuda")
    spc.spc_window_attn(q, k, v, o, window, sinks, lse, **kw)
    torch.cuda.synchronize()
    return q, k, v, o, lse


@pytest.mark.parametrize("lq,lk,Hq,Hkv", [(1, 300, 4, 1), (1, 9000, 32, 8), (40, 640, 8, 2), (300, 300, 8, 8), (1000, 1000, 8, 2),
                                          (900, 2311, 4, 1), (3, 200, 128, 1), (17, 130, 6, 2), (257, 257, 1, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 5), (63, 0), (64, 4), (65, 64), (128, 65), (127, 130), (200, 0),
                                          (1024, 4)])
def test_one_sequence(lq, lk, Hq, Hkv, window, sinks):
    q, k, v, o, lse = run_one(lq, lk, Hq, Hkv, window, sinks)
    check(o, lse, q, k, v, window_sight(lq, lk, window, sinks))


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 8, 9, 16, 17])
@pytest.mark.parametrize("Hkv", [1, 8])
@pytest.mark.parametrize("lk,window,sinks", [([1], 1, 0), ([15], 9, 3), ([16, 17, 0, 33], 16, 0), ([700, 64, 65, 1, 0, 5000], 300, 4),
                                             ([5000], 4000, 900), ([9000, 3], 5000, 1), ([260] * 40, 128, 1)])
def test_single_tokens(G, Hkv, lk, window, sinks):
    """One query token per sequence, of any number of heads over a KV head, in batches of one to many."""
    import bit_kv_cache_spc_gb300 as spc
    S, Hq, cap = len(lk), G * Hkv, max(lk) + 3
    q = rnd(1, S, 1, Hq, D)
    k, v = (rnd(i, S, Hkv, cap, D).transpose(1, 2) for i in (2, 3))
    o, lse = torch.full_like(q, 7.0), torch.full((S, 1, Hq), 7.0, device="cuda")
    for s, n in enumerate(lk):
        k[s, n:], v[s, n:] = math.nan, math.inf
    spc.spc_window_attn(q, k, v, o, window, sinks, lse, k_len=i32(lk))
    for s, n in enumerate(lk[:8]):
        check(o[s], lse[s], q[s], k[s, :n], v[s, :n], window_sight(1, n, window, sinks))


def test_single_tokens_of_some_sequences():
    """Packed single tokens between others' rows, empty sequences among them; keys of a row that a sequence does not have
    stay unread."""
    import bit_kv_cache_spc_gb300 as spc
    S, T, Hq, Hkv = 50, 900, 8, 2
    q, k, v = rnd(1, 2 * S, Hq, D), rnd(2, T, Hkv, D), rnd(3, T, Hkv, D)
    lk, kb, lq = [(s * 53) % 300 for s in range(S)], [(s * 31) % 600 for s in range(S)], [int(s % 5 != 2) for s in range(S)]
    o, lse = torch.full_like(q, 7.0), torch.full((2 * S, Hq), 7.0, device="cuda")
    spc.spc_window_attn(q, k, v, o, 100, 3, lse, q_begin=2 * torch.arange(S, dtype=torch.int32, device="cuda"), q_len=i32(lq),
                        k_begin=i32(kb), k_len=i32(lk), q_max=1, k_max=300)
    for s in range(S):
        b = 2 * s
        if lq[s]:
            check(o[b:b + 1], lse[b:b + 1], q[b:b + 1], k[kb[s]:kb[s] + lk[s]], v[kb[s]:kb[s] + lk[s]], window_sight(1, lk[s], 100, 3))
        assert bool((o[b + lq[s]:b + 2] == 7).all()) and bool((lse[b + lq[s]:b + 2] == 7).all())


@pytest.mark.parametrize("lq,lk,window,sinks", [(1, 0, 5, 2), (9, 4, 2, 1), (300, 130, 64, 10), (140, 1, 1, 0), (1300, 1100, 90, 5),
                                                (256, 100, 70, 200), (600, 345, 100, 0)])
def test_rows_that_see_nothing(lq, lk, window, sinks):
    q, k, v, o, lse = run_one(lq, lk, 4, 2, window, sinks)
    check(o, lse, q, k, v, window_sight(lq, lk, window, sinks))
    empty = lq - lk
    assert bool((o[:empty] == 0).all()) and bool((lse[:empty] == -math.inf).all())


@pytest.mark.parametrize("lq,lk,window", [(70, 70, 70), (70, 70, 1 << 30), (1, 3000, 3000), (300, 800, 2 ** 31 - 1)])
@pytest.mark.parametrize("sinks", [0, 3, 1 << 30])
def test_a_window_over_all_keys_is_the_plain_attention(lq, lk, window, sinks):
    import bit_kv_cache_spc_gb300 as spc
    q, k, v, o, lse = run_one(lq, lk, 4, 2, window, sinks)
    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
    spc.spc_prompt_attn(q, k, v, o2, lse2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("lq,lk,window", [(100, 1000, 64), (1, 5000, 700), (400, 400, 33)])
def test_first_tokens_up_to_all(lq, lk, window):
    """So many first tokens that the two runs of keys meet, or that they are all."""
    for sinks in (lk - window - 70, lk - window, lk, 1 << 30):
        q, k, v, o, lse = run_one(lq, lk, 4, 1, window, max(sinks, 0))
        check(o, lse, q, k, v, window_sight(lq, lk, window, max(sinks, 0)))


@pytest.mark.parametrize("mul", [12.0, 0.0])
@pytest.mark.parametrize("lq,lk", [(140, 700), (1, 3000)])
def test_growing_and_equal_scores(lq, lk, mul):
    q, k, v, o, lse = run_one(lq, lk, 4, 2, 150, 7, mul=mul)
    check(o, lse, q, k, v, window_sight(lq, lk, 150, 7))


@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (6, 6), (16, 8)])
@pytest.mark.parametrize("window,sinks", [(50, 3), (128, 0), (130, 70)])
def test_packed_sequences_of_different_lengths(Hq, Hkv, window, sinks):
    """Packed views of a fused projection; gaps between sequences keep their bytes."""
    import bit_kv_cache_spc_gb300 as spc
    lens = [37, 0, 1, 300, 128, 64]
    begin, T = [], 3
    for n in lens:
        begin.append(T)
        T += n + 2
    qkv = rnd(9, T, Hq + 2 * Hkv, D)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    o = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    spc.spc_window_attn(q, k, v, o, window, sinks, lse, q_begin=i32(begin), q_len=i32(lens), k_begin=i32(begin), k_len=i32(lens),
                        q_max=300, k_max=300)
    untouched = torch.ones(T, dtype=torch.bool, device="cuda")
    for b, n in zip(begin, lens):
        if n:
            check(o[b:b + n], lse[b:b + n], q[b:b + n], k[b:b + n], v[b:b + n], window_sight(n, n, window, sinks))
        untouched[b:b + n] = False
    assert bool((o[untouched] == 7).all()) and bool((lse[untouched] == 7).all())


@pytest.mark.parametrize("lq,lk", [([1, 1, 1], [500, 7, 1300]), ([20, 3, 0], [20, 700, 9]), ([130, 64, 1], [130, 900, 1]),
                                   ([1, 0, 1, 1], [0, 4000, 4000, 129])])
@pytest.mark.parametrize("window,sinks", [(100, 4), (1000, 100)])
def test_batch_over_head_major_caches(lq, lk, window, sinks):
    import bit_kv_cache_spc_gb300 as spc
    Hq, Hkv, cap = 8, 2, max(lk) + 5
    q = rnd(1, len(lq), max(lq), Hq, D)
    kb, vb = rnd(2, len(lq), Hkv, cap, D), rnd(3, len(lq), Hkv, cap, D)
    k, v = kb.transpose(1, 2), vb.transpose(1, 2)
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    spc.spc_window_attn(q, k, v, o, window, sinks, lse, q_len=i32(lq), k_len=i32(lk), k_max=max(lk))
    for s, (n, m) in enumerate(zip(lq, lk)):
        if n:
            check(o[s, :n], lse[s, :n], q[s, :n], k[s, :m], v[s, :m], window_sight(n, m, window, sinks))
        assert bool((o[s, n:] == 7).all()) and bool((lse[s, n:] == 7).all())


@pytest.mark.parametrize("lq,lk,G,window,sinks", [(200, 200, 2, 33, 5), (40, 1300, 4, 200, 70), (1, 900, 4, 100, 3), (1, 9000, 4, 5000, 3),
                                                  (600, 600, 1, 130, 0)])
@pytest.mark.parametrize("what", ["nan", "inf", "-inf", "lowest"])
def test_what_no_query_sees_does_not_matter(lq, lk, G, window, sinks, what):
    """Keys and values between the first tokens and the first window, and behind the sequence, hold infinities and NaN: the
    outputs are bit for bit those of harmless values there."""
    import bit_kv_cache_spc_gb300 as spc
    x = {"nan": math.nan, "inf": math.inf, "-inf": -math.inf, "lowest": torch.finfo(torch.bfloat16).min}[what]
    q, k, v = rnd(1, lq, 2 * G, D), rnd(2, lk + 200, 2, D), rnd(3, lk + 200, 2, D)
    seen = window_sight(lq, lk, window, sinks)
    dead = torch.ones(lk + 200, dtype=torch.bool, device="cuda")
    dead[:lk] = ~seen.any(0)
    outs = []
    for poison in (0.0, x):
        kk, vv = k.clone(), v.clone()
        kk[dead], vv[dead] = poison, poison
        o, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
        spc.spc_window_attn(q, kk, vv, o, window, sinks, lse, k_len=i32([lk]), k_max=lk + 100)
        outs.append((o, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    check(*outs[0], q, k[:lk], v[:lk], seen)


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_what_some_queries_see_does_not_matter_to_the_others(what):
    """A poisoned stretch of keys and values leaves the queries whose windows lie before or behind it as they were."""
    import bit_kv_cache_spc_gb300 as spc
    L, window, sinks = 700, 90, 5
    q, k, v = rnd(1, L, 4, D), rnd(2, L, 2, D), rnd(3, L, 2, D)
    o, lse = torch.zeros_like(q), torch.zeros((L, 4), device="cuda")
    spc.spc_window_attn(q, k, v, o, window, sinks, lse)
    k[301:340], v[301:340] = what, what
    o2, lse2 = torch.zeros_like(q), torch.zeros((L, 4), device="cuda")
    spc.spc_window_attn(q, k, v, o2, window, sinks, lse2)
    clean = ~window_sight(L, L, window, sinks)[:, 301:340].any(1)
    assert int(clean.sum()) == L - 39 - 89
    assert torch.equal(o[clean], o2[clean]) and torch.equal(lse[clean], lse2[clean])


def test_visible_infinities_and_nan():
    """Non-finite values of keys that a query sees reach its output with their sign, of first tokens, of window edges and
    of blocks that all rows see."""
    import bit_kv_cache_spc_gb300 as spc
    L, window, sinks = 500, 180, 9
    q, k, v = rnd(1, L, 2, D, mul=0.1), rnd(2, L, 1, D, mul=0.1), rnd(3, L, 1, D)
    places = {5: (3, math.inf), 130: (7, -math.inf), 260: (9, math.nan), 300: (11, math.inf), 8: (13, math.nan)}
    for j, (c, x) in places.items():
        v[j, 0, c] = x
    o = torch.zeros_like(q)
    spc.spc_window_attn(q, k, v, o, window, sinks)
    seen = window_sight(L, L, window, sinks)
    for j, (c, x) in places.items():
        s = seen[:, j]
        assert bool(torch.isfinite(o[~s][:, :, c]).all())
        got = o[s][:, :, c]
        assert bool(torch.isnan(got).all() if math.isnan(x) else (got == x).all())
    kept = [c for c in range(D) if c not in (3, 7, 9, 11, 13)]
    o2 = torch.zeros_like(q)
    spc.spc_window_attn(q, k, torch.where(torch.isfinite(v), v, torch.zeros_like(v)), o2, window, sinks)
    assert torch.equal(o[:, :, kept], o2[:, :, kept])


@pytest.mark.parametrize("S,most", [(40, 700), (256, 300), (300, 300)])
def test_many_packed_sequences(S, most):
    import bit_kv_cache_spc_gb300 as spc
    lens = [(s * 97) % 41 if s % 13 else (most if s == 0 else most // (1 + s % 7)) for s in range(S)]
    begin = [sum(lens[:s]) for s in range(S)]
    T, Hq, Hkv = sum(lens), 2, 1
    q, k, v = rnd(1, T, Hq, D), rnd(2, T, Hkv, D), rnd(3, T, Hkv, D)
    o, lse = torch.full_like(q, 7.0), torch.full((T, Hq), 7.0, device="cuda")
    spc.spc_window_attn(q, k, v, o, 77, 2, lse, q_begin=i32(begin), q_len=i32(lens), k_begin=i32(begin), k_len=i32(lens),
                        q_max=most, k_max=most)
    assert not bool((lse == 7).any())
    for s in list(range(0, S, 13)) + [1, 2, S - 1]:
        b, n = begin[s], lens[s]
        if n:
            check(o[b:b + n], lse[b:b + n], q[b:b + n], k[b:b + n], v[b:b + n], window_sight(n, n, 77, 2))


def test_other_strides_and_scale():
    import bit_kv_cache_spc_gb300 as spc
    L, Hq, Hkv = 150, 4, 2
    q = rnd(1, Hq, 2 * L, D)[:, ::2].transpose(0, 1)
    k = rnd(2, L, Hkv, 2, D)[:, :, 1]
    v = rnd(3, Hkv, L, 3 * D)[:, :, D:2 * D].transpose(0, 1)
    ob = torch.full((Hq, L, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    spc.spc_window_attn(q, k, v, ob[:, :, D:].transpose(0, 1), 40, 1, scale=0.03)
    check(ob[:, :, D:].transpose(0, 1), None, q, k, v, window_sight(L, L, 40, 1), 0.03)
    assert bool((ob[:, :, :D] == 7).all())


def test_device_lengths_are_held_to_the_tensors():
    import bit_kv_cache_spc_gb300 as spc
    T, Hq, Hkv = 100, 4, 2
    q, k, v = rnd(1, T, Hq, D), rnd(2, T, Hkv, D), rnd(3, T, Hkv, D)
    buf = torch.full((T + 300, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    o = buf[150:150 + T]
    spc.spc_window_attn(q, k, v, o, 9, 2, q_begin=i32([-5, 90]), q_len=i32([30, 1000]), k_begin=i32([0, 80]),
                        k_len=i32([30, 1 << 30]), q_max=40, k_max=60)
    check(o[:30], None, q[:30], k[:30], v[:30], window_sight(30, 30, 9, 2))
    check(o[90:], None, q[90:], k[80:], v[80:], window_sight(10, 20, 9, 2))
    assert bool((buf[:150] == 7).all()) and bool((buf[150 + 30:150 + 90] == 7).all()) and bool((buf[150 + T:] == 7).all())


@pytest.mark.parametrize("lq", [1, 2])
def test_graphs_and_streams_repeat_the_same_bits(lq):
    """Captured and replayed with other lengths, on other streams, two calls at once with their own workspaces."""
    import bit_kv_cache_spc_gb300 as spc
    q, k, v = rnd(1, lq, 32, D), rnd(2, 9000, 8, D), rnd(3, 9000, 8, D)
    o, lse, n = torch.zeros_like(q), torch.zeros((lq, 32), device="cuda"), i32([9000])
    need = spc.spc_window_attn_workspace_bytes(q, k, v, o, 4000, 4)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    assert (need > 256) == (lq == 2)  # two queries over a long window: the keys are split
    spc.spc_window_attn(q, k, v, o, 4000, 4, lse, k_len=n, ws=ws)
    want = (o.clone(), lse.clone())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        spc.spc_window_attn(q, k, v, o, 4000, 4, lse, k_len=n, ws=ws)
    o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    n.fill_(5003)
    g.replay()
    torch.cuda.synchronize()
    check(o, lse, q, k[:5003], v[:5003], window_sight(lq, 5003, 4000, 4))
    n.fill_(9000)
    side = [torch.cuda.Stream() for _ in range(2)]
    outs, wss = [torch.zeros_like(o) for _ in side], [torch.zeros_like(ws) for _ in side]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, x, w in zip(side, outs, wss):
            spc.spc_window_attn(q, k, v, x, 4000, 4, k_len=n, ws=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[0]) for x in outs)
    assert spc.spc_prompt_attn_status(ws) == 0 and spc.spc_prompt_attn_status() == 0


def test_a_wait_that_runs_out_is_reported():
    """With a limit of a nanosecond, over windows of half a million keys without a split; the next call is right."""
    import bit_kv_cache_spc_gb300 as spc
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    z = dict(dtype=torch.bfloat16, device="cuda")
    q, k = torch.zeros((2 * sms, 128, D), **z), torch.zeros((1 << 19, 1, D), **z)
    v, o, ws = torch.ones_like(k), torch.full_like(q, 7.0), torch.zeros(256, dtype=torch.uint8, device="cuda")
    window = (1 << 19) - 1
    assert spc.spc_window_attn_workspace_bytes(q, k, v, o, window) == 256
    before = spc.spc_prompt_attn_wait_limit(1)
    try:
        spc.spc_window_attn(q, k, v, o, window, ws=ws)
        spc.spc_prompt_attn_wait_limit(before)
        assert spc.spc_prompt_attn_status(ws) == 6 and spc.spc_prompt_attn_status(ws) == 0
        assert spc.spc_prompt_attn_status() == 6 and spc.spc_prompt_attn_status() == 0
        spc.spc_window_attn(q, k, v, o, window, ws=ws)
        assert bool((o == 1).all()) and spc.spc_prompt_attn_status(ws) == 0
    finally:
        spc.spc_prompt_attn_wait_limit(before)
        spc.spc_prompt_attn_status()
