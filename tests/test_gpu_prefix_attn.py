"""The attention of sequences that share a prefix (spc_prefix_attn) against a plain 64-bit form."""
import math

import pytest
import torch

from sight_ref import check, i32, prefix_sight, rnd

pytestmark = pytest.mark.gpu
D = 128


def both(pk, k):
    return torch.cat([pk, k])


@pytest.mark.parametrize("P", [1, 63, 64, 65, 127, 130, 2003, 9000])
@pytest.mark.parametrize("lq,lk,Hq,Hkv", [(1, 1, 4, 1), (1, 300, 4, 2), (5, 5, 1, 1), (40, 170, 8, 2), (130, 130, 6, 2), (300, 300, 4, 4),
                                          (3, 70, 128, 1), (257, 400, 2, 1)])
def test_one_sequence(P, lq, lk, Hq, Hkv):
    import bit_kv_cache_spc_gb300 as spc
    q, k, v = rnd(0, lq, Hq, D), rnd(1, lk, Hkv, D), rnd(2, lk, Hkv, D)
    pk, pv = rnd(3, P, Hkv, D), rnd(4, P, Hkv, D)
    o, lse = torch.full_like(q, 7.0), torch.full((lq, Hq), 7.0, device="cuda")
    spc.spc_prefix_attn(q, pk, pv, k, v, o, lse)
    check(o, lse, q, both(pk, k), both(pv, v), prefix_sight(lq, lk, P))


@pytest.mark.parametrize("lq,lk", [(1, 0), (9, 4), (300, 130), (140, 1), (200, 0)])
@pytest.mark.parametrize("P", [5, 200, 3000])
def test_rows_without_a_key_of_their_own(lq, lk, P):
    """They see the prefix alone."""
    import bit_kv_cache_spc_gb300 as spc
    q, k, v = rnd(0, lq, 4, D), rnd(1, lk, 2, D), rnd(2, lk, 2, D)
    pk, pv = rnd(3, P, 2, D), rnd(4, P, 2, D)
    o, lse = torch.full_like(q, 7.0), torch.full((lq, 4), 7.0, device="cuda")
    spc.spc_prefix_attn(q, pk, pv, k, v, o, lse)
    check(o, lse, q, both(pk, k), both(pv, v), prefix_sight(lq, lk, P))


@pytest.mark.parametrize("lq,lk", [(1, 2000), (70, 70), (9, 4)])
def test_an_empty_prefix_is_the_plain_attention(lq, lk):
    """Of no tokens: its bits; of a length of zero on the device: its values, and rows that see nothing."""
    import bit_kv_cache_spc_gb300 as spc
    q, k, v, p = rnd(0, lq, 4, D), rnd(1, lk, 2, D), rnd(2, lk, 2, D), rnd(3, 100, 2, D)
    o, lse = torch.zeros_like(q), torch.zeros((lq, 4), device="cuda")
    o2, lse2 = torch.zeros_like(q), torch.zeros((lq, 4), device="cuda")
    spc.spc_prompt_attn(q, k, v, o, lse)
    spc.spc_prefix_attn(q, p[:0], p[:0], k, v, o2, lse2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    p.fill_(math.nan)
    spc.spc_prefix_attn(q, p, p, k, v, o2, lse2, p_len=i32([0]))
    check(o2, lse2, q, k, v, prefix_sight(lq, lk, 0))
    if lq > lk:
        assert bool((o2[:lq - lk] == 0).all()) and bool((lse2[:lq - lk] == -math.inf).all())


@pytest.mark.parametrize("lq", [1, 150])
@pytest.mark.parametrize("n,cap", [(70, 300), (128, 129), (1, 64), (2000, 5000), (5000, 5000), (9999, 5000), (-3, 50)])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_the_length_of_the_prefix_on_the_device(lq, n, cap, what):
    """Rows behind it do not matter, whatever they hold; a length beyond the tensor is held to it."""
    import bit_kv_cache_spc_gb300 as spc
    q, k, v, pk, pv = rnd(0, lq, 8, D), rnd(1, 200, 2, D), rnd(2, 200, 2, D), rnd(3, cap, 2, D), rnd(4, cap, 2, D)
    P = max(0, min(n, cap))
    pk[P:], pv[P:] = what, what
    o, lse = torch.zeros_like(q), torch.zeros((lq, 8), device="cuda")
    spc.spc_prefix_attn(q, pk, pv, k, v, o, lse, p_len=i32([n]))
    check(o, lse, q, both(pk[:P], k), both(pv[:P], v), prefix_sight(lq, 200, P))


@pytest.mark.parametrize("P", [50, 700, 4001])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (6, 6), (16, 8)])
@pytest.mark.parametrize("lens", [[37, 0, 1, 300, 128, 64], [1, 1, 1, 0, 1, 1, 1], [5, 9, 1, 1, 30, 2, 0, 3, 3, 17, 40, 1]])
def test_packed_sequences_of_different_lengths(P, Hq, Hkv, lens):
    """Packed views of a fused projection; gaps between sequences keep their bytes, whatever their queries hold."""
    import bit_kv_cache_spc_gb300 as spc
    begin, T = [], 3
    for n in lens:
        begin.append(T)
        T += n + 2
    qkv = rnd(9, T, Hq + 2 * Hkv, D)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    pk, pv = rnd(3, P, Hkv, D), rnd(4, P, Hkv, D)
    o = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    untouched = torch.ones(T, dtype=torch.bool, device="cuda")
    for b, n in zip(begin, lens):
        untouched[b:b + n] = False
    qkv[untouched] = math.nan
    spc.spc_prefix_attn(q, pk, pv, k, v, o, lse, q_begin=i32(begin), q_len=i32(lens), k_begin=i32(begin), k_len=i32(lens),
                        q_max=max(lens), k_max=max(lens))
    for b, n in zip(begin, lens):
        if n:
            check(o[b:b + n], lse[b:b + n], q[b:b + n], both(pk, k[b:b + n]), both(pv, v[b:b + n]), prefix_sight(n, n, P))
    assert bool((o[untouched] == 7).all()) and bool((lse[untouched] == 7).all())


@pytest.mark.parametrize("P", [300, 5000])
@pytest.mark.parametrize("lq,lk", [([1, 1, 1], [500, 7, 1300]), ([1] * 70, [(s * 37) % 90 for s in range(70)]), ([20, 3, 0], [20, 700, 9]),
                                   ([130, 64, 1], [130, 900, 1]), ([1, 0, 1, 1], [0, 400, 400, 129]), ([2, 5, 3, 0, 5, 1], [2, 50, 33, 9, 5, 0])])
def test_batch_over_head_major_caches(P, lq, lk):
    """A padded batch of queries over cache buffers [S][Hkv][cap][D], a prefix in such a buffer too."""
    import bit_kv_cache_spc_gb300 as spc
    Hq, Hkv, cap = 8, 2, max(lk) + 5
    q = rnd(1, len(lq), max(lq), Hq, D)
    k, v = (rnd(i, len(lq), Hkv, cap, D).transpose(1, 2) for i in (2, 3))
    pk, pv = (rnd(i, Hkv, P + 9, D)[:, :P].transpose(0, 1) for i in (4, 5))
    for s, n in enumerate(lq):
        q[s, n:] = math.nan
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    spc.spc_prefix_attn(q, pk, pv, k, v, o, lse, q_len=i32(lq), k_len=i32(lk), k_max=max(lk))
    for s, (n, m) in enumerate(zip(lq, lk)):
        if n:
            check(o[s, :n], lse[s, :n], q[s, :n], both(pk, k[s, :m]), both(pv, v[s, :m]), prefix_sight(n, m, P))
        assert bool((o[s, n:] == 7).all()) and bool((lse[s, n:] == 7).all())


@pytest.mark.parametrize("S,G", [(1, 4), (33, 4), (64, 1), (200, 2), (600, 4), (17, 32)])
def test_single_tokens_of_many_sequences(S, G):
    """Packed single tokens, some of the sequences sharing keys of their own too."""
    import bit_kv_cache_spc_gb300 as spc
    T, Hkv, P = 900, 2, 1111
    Hq = G * Hkv
    q, k, v, pk, pv = rnd(1, S, Hq, D), rnd(2, T, Hkv, D), rnd(3, T, Hkv, D), rnd(4, P, Hkv, D), rnd(5, P, Hkv, D)
    lk = [(s * 53) % 300 for s in range(S)]
    kb = [(s * 31) % 600 for s in range(S)]
    o, lse = torch.zeros_like(q), torch.zeros((S, Hq), device="cuda")
    spc.spc_prefix_attn(q, pk, pv, k, v, o, lse, q_begin=torch.arange(S, dtype=torch.int32, device="cuda"), k_begin=i32(kb),
                        k_len=i32(lk), q_max=1, k_max=300)
    for s in range(0, S, 7):
        at = slice(kb[s], kb[s] + lk[s])
        check(o[s:s + 1], lse[s:s + 1], q[s:s + 1], both(pk, k[at]), both(pv, v[at]), prefix_sight(1, lk[s], P))


def test_without_keys_of_their_own():
    """Keys and values of no tokens: the prefix alone."""
    import bit_kv_cache_spc_gb300 as spc
    q, pk, pv = rnd(1, 5, 3, 8, D), rnd(4, 700, 2, D), rnd(5, 700, 2, D)
    none = torch.empty((5, 0, 2, D), dtype=torch.bfloat16, device="cuda")
    o, lse = torch.zeros_like(q), torch.zeros((5, 3, 8), device="cuda")
    spc.spc_prefix_attn(q, pk, pv, none, none, o, lse)
    for s in range(5):
        check(o[s], lse[s], q[s], pk, pv, prefix_sight(3, 0, 700))


@pytest.mark.parametrize("lq", [1, 130])
@pytest.mark.parametrize("mul", [12.0, 0.0])
def test_growing_and_equal_scores(lq, mul):
    import bit_kv_cache_spc_gb300 as spc
    q, k, v, pk, pv = rnd(1, lq, 4, D, mul=mul), rnd(2, 300, 2, D), rnd(3, 300, 2, D), rnd(4, 900, 2, D), rnd(5, 900, 2, D)
    o, lse = torch.zeros_like(q), torch.zeros((lq, 4), device="cuda")
    spc.spc_prefix_attn(q, pk, pv, k, v, o, lse)
    check(o, lse, q, both(pk, k), both(pv, v), prefix_sight(lq, 300, 900))


@pytest.mark.parametrize("lq,P", [(1, 900), (200, 100), (40, 3000)])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_masked_places_do_not_matter(lq, P, what):
    """Own keys and values behind the first half of the queries are poisoned: that half keeps its bits."""
    import bit_kv_cache_spc_gb300 as spc
    lk = 200 + lq
    q, k, v, pk, pv = rnd(1, lq, 4, D), rnd(2, lk + 90, 2, D), rnd(3, lk + 90, 2, D), rnd(4, P, 2, D), rnd(5, P, 2, D)
    cut = lk - lq // 2
    outs = []
    for poison in (0.0, what):
        kk, vv = k.clone(), v.clone()
        kk[cut:], vv[cut:] = poison, poison
        o, lse = torch.zeros_like(q), torch.zeros((lq, 4), device="cuda")
        spc.spc_prefix_attn(q, pk, pv, kk, vv, o, lse, k_len=i32([lk]))
        outs.append((o, lse))
    clean = lq - lq // 2
    assert torch.equal(outs[0][0][:clean], outs[1][0][:clean]) and torch.equal(outs[0][1][:clean], outs[1][1][:clean])


@pytest.mark.parametrize("S", [1, 40])
def test_visible_infinities_and_nan(S):
    """Of the prefix, in its last, partial block too, and of a sequence's own keys."""
    import bit_kv_cache_spc_gb300 as spc
    L, P = 7, 200
    q, k, v = rnd(1, S, L, 2, D, mul=0.1), rnd(2, S, 90, 1, D, mul=0.1), rnd(3, S, 90, 1, D)
    pk, pv = rnd(4, P, 1, D, mul=0.1), rnd(5, P, 1, D)
    pv[10, 0, 3], pv[197, 0, 7], pv[199, 0, 9] = math.inf, -math.inf, math.nan
    v[0, 86, 0, 11], v[0, 30, 0, 13] = math.inf, -math.inf
    o = torch.zeros_like(q)
    spc.spc_prefix_attn(q, pk, pv, k, v, o)
    assert bool((o[..., 3] == math.inf).all()) and bool((o[..., 7] == -math.inf).all()) and bool(torch.isnan(o[..., 9]).all())
    assert bool((o[0, 3:, :, 11] == math.inf).all()) and bool(torch.isfinite(o[0, :3, :, 11]).all())
    assert bool((o[0, :, :, 13] == -math.inf).all()) and bool(torch.isfinite(o[1:, :, :, 13]).all())
    kept = [c for c in range(D) if c not in (3, 7, 9, 11, 13)]
    o2, zero = torch.zeros_like(q), lambda x: torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    spc.spc_prefix_attn(q, pk, zero(pv), k, zero(v), o2)
    assert torch.equal(o[..., kept], o2[..., kept])


@pytest.mark.parametrize("S,lq", [(1, 1), (24, 1), (3, 90)])
def test_graphs_and_streams_repeat_the_same_bits(S, lq):
    """Captured and replayed with another length of the prefix, on other streams, two calls at once with their own workspaces."""
    import bit_kv_cache_spc_gb300 as spc
    q, k, v = rnd(1, S, lq, 32, D), rnd(2, S, 200, 8, D), rnd(3, S, 200, 8, D)
    pk, pv, n = rnd(4, 5000, 8, D), rnd(5, 5000, 8, D), i32([5000])
    o, lse = torch.zeros_like(q), torch.zeros((S, lq, 32), device="cuda")
    ws = torch.zeros(spc.spc_prefix_attn_workspace_bytes(q, pk, pv, k, v, o), dtype=torch.uint8, device="cuda")
    spc.spc_prefix_attn(q, pk, pv, k, v, o, lse, p_len=n, ws=ws)
    want = (o.clone(), lse.clone())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        spc.spc_prefix_attn(q, pk, pv, k, v, o, lse, p_len=n, ws=ws)
    o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    n.fill_(777)
    g.replay()
    torch.cuda.synchronize()
    for s in range(0, S, 5):
        check(o[s], lse[s], q[s], both(pk[:777], k[s]), both(pv[:777], v[s]), prefix_sight(lq, 200, 777))
    n.fill_(5000)
    side = [torch.cuda.Stream() for _ in range(2)]
    outs, wss = [torch.zeros_like(o) for _ in side], [torch.zeros_like(ws) for _ in side]
    torch.cuda.synchronize()
    for _ in range(4):
        for st, x, w in zip(side, outs, wss):
            spc.spc_prefix_attn(q, pk, pv, k, v, x, p_len=n, ws=w, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[0]) for x in outs)
    spc.spc_prefix_attn(q, pk, pv, k, v, outs[0], p_len=n)  # its own workspace
    assert torch.equal(outs[0], want[0])
    assert spc.spc_prompt_attn_status(ws) == 0 and spc.spc_prompt_attn_status() == 0


def test_device_lengths_are_held_to_the_tensors():
    import bit_kv_cache_spc_gb300 as spc
    T, Hq, Hkv = 100, 4, 2
    q, k, v, pk, pv = rnd(1, T, Hq, D), rnd(2, T, Hkv, D), rnd(3, T, Hkv, D), rnd(4, 70, Hkv, D), rnd(5, 70, Hkv, D)
    buf = torch.full((T + 300, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    o = buf[150:150 + T]
    spc.spc_prefix_attn(q, pk, pv, k, v, o, q_begin=i32([-5, 90]), q_len=i32([30, 1000]), k_begin=i32([0, 80]),
                        k_len=i32([30, 1 << 30]), q_max=40, k_max=60)
    check(o[:30], None, q[:30], both(pk, k[:30]), both(pv, v[:30]), prefix_sight(30, 30, 70))
    check(o[90:], None, q[90:], both(pk, k[80:]), both(pv, v[80:]), prefix_sight(10, 20, 70))
    assert bool((buf[:150] == 7).all()) and bool((buf[150 + 30:150 + 90] == 7).all()) and bool((buf[150 + T:] == 7).all())


def test_a_wait_that_runs_out_is_reported():
    """With a limit of a nanosecond, over a prefix of half a million keys; the next call is right."""
    import bit_kv_cache_spc_gb300 as spc
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    z = dict(dtype=torch.bfloat16, device="cuda")
    q, pk, k = torch.zeros((2 * sms, 128, D), **z), torch.zeros((1 << 19, 1, D), **z), torch.zeros((2 * sms, 1, D), **z)
    pv, v, o = torch.ones_like(pk), torch.ones_like(k), torch.full_like(q, 7.0)
    ws = torch.zeros(spc.spc_prefix_attn_workspace_bytes(q, pk, pv, k, v, o), dtype=torch.uint8, device="cuda")
    before = spc.spc_prompt_attn_wait_limit(1)
    try:
        spc.spc_prefix_attn(q, pk, pv, k, v, o, ws=ws)
        spc.spc_prompt_attn_wait_limit(before)
        assert spc.spc_prompt_attn_status(ws) == 6 and spc.spc_prompt_attn_status(ws) == 0
        assert spc.spc_prompt_attn_status() == 6 and spc.spc_prompt_attn_status() == 0
        spc.spc_prefix_attn(q, pk, pv, k, v, o, ws=ws)
        assert bool((o == 1).all()) and spc.spc_prompt_attn_status(ws) == 0
    finally:
        spc.spc_prompt_attn_wait_limit(before)
        spc.spc_prompt_attn_status()


@pytest.mark.parametrize("P", [64, 1000, 8001])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (6, 2), (32, 1)])
@pytest.mark.parametrize("S,most,own", [(2, 20, 90), (17, 77, 0), (40, 9, 300), (64, 30, 33), (65, 30, 33), (64, 3, 0)])
def test_few_rows_each_of_many_sequences(P, Hq, Hkv, S, most, own):
    """Tiles with rows of several sequences, whose own keys lie anywhere, are shared, or do not reach all of their rows."""
    import bit_kv_cache_spc_gb300 as spc
    lq = [(s * 37) % (most + 1) if s else most for s in range(S)]
    lk = [(s * 53) % (own + 1) if own else lq[s] for s in range(S)]
    T, N = sum(lq) + 5, 700
    q, k, v, pk, pv = rnd(1, T, Hq, D), rnd(2, N, Hkv, D), rnd(3, N, Hkv, D), rnd(4, P, Hkv, D), rnd(5, P, Hkv, D)
    qb = [sum(lq[:s]) + 3 * (s > S // 2) for s in range(S)]  # a gap within
    kb = [(s * 131) % (N - max(lk) + 1) for s in range(S)]
    o, lse = torch.full_like(q, 7.0), torch.full((T, Hq), 7.0, device="cuda")
    spc.spc_prefix_attn(q, pk, pv, k, v, o, lse, q_begin=i32(qb), q_len=i32(lq), k_begin=i32(kb), k_len=i32(lk), q_max=most,
                        k_max=max(max(lk), 1))
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    for s in range(S):
        rest[qb[s]:qb[s] + lq[s]] = False
        if lq[s] and (s % 5 == 0 or S < 20):
            at, own_k = slice(qb[s], qb[s] + lq[s]), slice(kb[s], kb[s] + lk[s])
            check(o[at], lse[at], q[at], both(pk, k[own_k]), both(pv, v[own_k]), prefix_sight(lq[s], lk[s], P))
    assert bool((o[rest] == 7).all()) and bool((lse[rest] == 7).all()) and not bool((lse[~rest] == 7).any())


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("S,n", [(6, 20), (40, 7)])
def test_other_sequences_keys_do_not_matter(S, n, what):
    """One sequence's own keys and values are poisoned: the others, in the same tiles, keep their bits; so do its own rows
    before the poisoned place."""
    import bit_kv_cache_spc_gb300 as spc
    P, Hq, Hkv = 500, 4, 2
    q, k, v, pk, pv = rnd(1, S * n, Hq, D), rnd(2, S * n, Hkv, D), rnd(3, S * n, Hkv, D), rnd(4, P, Hkv, D), rnd(5, P, Hkv, D)
    at = i32([s * n for s in range(S)])
    outs = []
    for x in (0.0, what):
        kk, vv = k.clone(), v.clone()
        kk[2 * n + 4:3 * n], vv[2 * n + 4:3 * n] = x, x
        o, lse = torch.zeros_like(q), torch.zeros((S * n, Hq), device="cuda")
        spc.spc_prefix_attn(q, pk, pv, kk, vv, o, lse, q_begin=at, q_len=i32([n] * S), k_begin=at, k_len=i32([n] * S), q_max=n, k_max=n)
        outs.append((o, lse))
    clean = torch.ones(S * n, dtype=torch.bool, device="cuda")
    clean[2 * n + 4:3 * n] = False
    assert torch.equal(outs[0][0][clean], outs[1][0][clean]) and torch.equal(outs[0][1][clean], outs[1][1][clean])


def test_visible_infinities_and_nan_of_one_sequence_among_others():
    import bit_kv_cache_spc_gb300 as spc
    S, n, P, Hq, Hkv = 9, 13, 200, 2, 1
    q, k, v = rnd(1, S * n, Hq, D, mul=0.1), rnd(2, S * n, Hkv, D, mul=0.1), rnd(3, S * n, Hkv, D)
    pk, pv = rnd(4, P, Hkv, D, mul=0.1), rnd(5, P, Hkv, D)
    v[3 * n + 5, 0, 3], v[7 * n, 0, 9], pv[198, 0, 20] = math.inf, math.nan, -math.inf
    at, o = i32([s * n for s in range(S)]), torch.zeros_like(q)
    spc.spc_prefix_attn(q, pk, pv, k, v, o, q_begin=at, q_len=i32([n] * S), k_begin=at, k_len=i32([n] * S), q_max=n, k_max=n)
    three, seven = slice(3 * n + 5, 4 * n), slice(7 * n, 8 * n)
    rest = torch.ones(S * n, dtype=torch.bool, device="cuda")
    rest[three], rest[seven] = False, False
    assert bool((o[three, :, 3] == math.inf).all()) and bool(torch.isnan(o[seven, :, 9]).all()) and bool((o[..., 20] == -math.inf).all())
    assert bool(torch.isfinite(o[rest][:, :, [c for c in range(D) if c != 20]]).all())
