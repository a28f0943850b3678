"""The causal attention of prompts (spc_prompt_attn) against a plain 64-bit form."""
import math

import pytest
import torch

from prompt_ref import attention

pytestmark = pytest.mark.gpu
D = 128


def rnd(seed, *shape, mul=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * mul).to(torch.bfloat16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check(got_o, got_lse, q, k, v, scale=None):
    """One sequence's output rows against the 64-bit form."""
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    o, lse, o_tol, lse_tol = attention(q, k, v, scale)
    err = (got_o.double() - o).abs()
    assert bool((err <= o_tol).all()), f"o off by {float((err - o_tol).max())} beyond the bound"
    if got_lse is not None:
        none = torch.isinf(lse)
        assert torch.equal(torch.isinf(got_lse) & (got_lse < 0), none)
        err = (got_lse.double() - lse)[~none].abs()
        assert bool((err <= lse_tol[~none]).all())


def run_one(lq, lk, Hq, Hkv, seed=0, mul=1.0, **kw):
    import bit_kv_cache_spc_gb300 as spc
    q, k, v = rnd(seed, lq, Hq, D, mul=mul), rnd(seed + 1, lk, Hkv, D), rnd(seed + 2, lk, Hkv, D)
    o = torch.full((lq, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((lq, Hq), 7.0, device="cuda")
    spc.spc_prompt_attn(q, k, v, o, lse, **kw)
    torch.cuda.synchronize()
    return q, k, v, o, lse


@pytest.mark.parametrize("lq,lk,Hq,Hkv", [
    (1, 1, 1, 1), (128, 128, 1, 1), (5, 5, 4, 1), (64, 64, 4, 2), (1, 300, 4, 1), (129, 129, 2, 2), (32, 128, 4, 1),
    (33, 161, 4, 1), (256, 256, 1, 1), (257, 257, 1, 1), (40, 640, 8, 2), (17, 130, 6, 2), (9, 77, 7, 1),
    (70, 70, 16, 1), (3, 200, 128, 1), (200, 333, 4, 4), (1, 2048, 4, 1), (2, 1537, 32, 8), (300, 300, 8, 8),
    (300, 300, 4, 2), (1, 1, 32, 8), (1000, 1000, 8, 2), (900, 2311, 4, 1), (130, 5000, 8, 2), (1, 9000, 32, 8)])
def test_one_sequence(lq, lk, Hq, Hkv):
    q, k, v, o, lse = run_one(lq, lk, Hq, Hkv)
    check(o, lse, q, k, v)


@pytest.mark.parametrize("lq,lk,most,Hq,Hkv", [(1300, 4096, 4096, 16, 16), (1300, 4031, 4096, 16, 16),
                                               (1300, 1700, 4096, 16, 16), (1300, 900, 4096, 16, 16),
                                               (1300, 0, 4096, 16, 16), (333, 12000, 12000, 28, 4)])
def test_a_last_split_shorter_than_the_others(lq, lk, most, Hq, Hkv):
    """More items than half of the SMs: on 152, two to four splits of which the last ones run in turn."""
    import bit_kv_cache_spc_gb300 as spc
    q, k, v = rnd(1, lq, Hq, D), rnd(2, most, Hkv, D), rnd(3, most, Hkv, D)
    k[lk:], v[lk:] = math.nan, math.nan
    o = torch.full((lq, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((lq, Hq), 7.0, device="cuda")
    spc.spc_prompt_attn(q, k, v, o, lse, k_len=i32([lk]))
    check(o, lse, q, k[:lk], v[:lk])


@pytest.mark.parametrize("lq,lk,G", [(1, 0, 2), (7, 0, 2), (9, 4, 2), (300, 130, 2), (140, 1, 2), (1300, 1100, 2),
                                     (256, 100, 1), (256, 128, 1), (300, 290, 1), (600, 345, 1), (200, 72, 1)])
def test_rows_that_see_nothing(lq, lk, G):
    """Also whole tiles of such rows beside one that sees something."""
    q, k, v, o, lse = run_one(lq, lk, 2 * G, 2)
    check(o, lse, q, k, v)
    empty = lq - lk
    assert bool((o[:empty] == 0).all()) and bool((lse[:empty] == -math.inf).all())


@pytest.mark.parametrize("mul", [12.0, 0.0])
@pytest.mark.parametrize("lq,lk", [(140, 700), (1, 3000)])
def test_growing_and_equal_scores(lq, lk, mul):
    """Scores over hundreds (the running maximum moves often) and all-equal ones."""
    q, k, v, o, lse = run_one(lq, lk, 4, 2, mul=mul)
    check(o, lse, q, k, v)


@pytest.mark.parametrize("lq", [1, 130])
def test_scores_that_grow_along_the_keys(lq):
    """Each key tile raises the maximum beyond the slack, so O is rescaled every time."""
    import bit_kv_cache_spc_gb300 as spc
    q, k, v = rnd(3, lq, 2, D).abs(), rnd(4, 900, 1, D).abs(), rnd(5, 900, 1, D)
    k = (k * torch.linspace(0.1, 3.0, 900, device="cuda")[:, None, None]).to(torch.bfloat16)
    o, lse = torch.zeros_like(q), torch.zeros((lq, 2), device="cuda")
    spc.spc_prompt_attn(q, k, v, o, lse)
    check(o, lse, q, k, v)


@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (6, 6), (16, 8)])
def test_packed_sequences_of_different_lengths(Hq, Hkv):
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
    spc.spc_prompt_attn(q, k, v, o, lse, q_begin=i32(begin), q_len=i32(lens), k_begin=i32(begin), k_len=i32(lens),
                        q_max=300, k_max=300)
    untouched = torch.ones(T, dtype=torch.bool, device="cuda")
    for b, n in zip(begin, lens):
        if n:
            check(o[b:b + n], lse[b:b + n], q[b:b + n], k[b:b + n], v[b:b + n])
        untouched[b:b + n] = False
    assert bool((o[untouched] == 7).all()) and bool((lse[untouched] == 7).all())


@pytest.mark.parametrize("lq,lk", [([1, 1, 1], [500, 7, 1300]), ([20, 3, 0], [20, 700, 9]), ([130, 64, 1], [130, 900, 1]),
                                   ([1, 0, 1, 1], [0, 4000, 4000, 129])])
def test_batch_over_head_major_caches(lq, lk):
    """A padded batch of queries over cache buffers [S][Hkv][cap][D] (few rows: the keys are split)."""
    import bit_kv_cache_spc_gb300 as spc
    Hq, Hkv, cap = 8, 2, max(lk) + 5
    q = rnd(1, len(lq), max(lq), Hq, D)
    kb, vb = rnd(2, len(lq), Hkv, cap, D), rnd(3, len(lq), Hkv, cap, D)
    k, v = kb.transpose(1, 2), vb.transpose(1, 2)
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    spc.spc_prompt_attn(q, k, v, o, lse, q_len=i32(lq), k_len=i32(lk), k_max=max(lk))
    for s, (n, m) in enumerate(zip(lq, lk)):
        if n:
            check(o[s, :n], lse[s, :n], q[s, :n], k[s, :m], v[s, :m])
        assert bool((o[s, n:] == 7).all()) and bool((lse[s, n:] == 7).all())


@pytest.mark.parametrize("lq,lk,G", [(200, 200, 2), (40, 1300, 4), (1, 900, 4)])
@pytest.mark.parametrize("what", ["nan", "inf", "-inf", "lowest"])
def test_masked_places_do_not_matter(lq, lk, G, what):
    """Rows behind the sequence and keys and values that a query does not see hold infinities and NaN: the outputs
    are bit for bit those of harmless values there."""
    import bit_kv_cache_spc_gb300 as spc
    x = {"nan": math.nan, "inf": math.inf, "-inf": -math.inf, "lowest": torch.finfo(torch.bfloat16).min}[what]
    q, k, v = rnd(1, lq, 2 * G, D), rnd(2, lk + 200, 2, D), rnd(3, lk + 200, 2, D)
    cut = lk - lq // 2 if lq > 1 else lk  # the last half of the queries sees poisoned keys, the first does not
    outs = []
    for poison in (0.0, x):
        kk, vv = k.clone(), v.clone()
        kk[cut:], vv[cut:] = poison, poison
        o, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
        spc.spc_prompt_attn(q, kk, vv, o, lse, k_len=i32([lk]), k_max=lk + 100)
        outs.append((o, lse))
    clean = lq - (lk - cut)
    assert torch.equal(outs[0][0][:clean], outs[1][0][:clean]) and torch.equal(outs[0][1][:clean], outs[1][1][:clean])
    check(outs[1][0][:clean], outs[1][1][:clean], q[:clean], k[:cut], v[:cut])


def test_visible_infinities_and_nan():
    """Non-finite values of keys that a query sees reach its output with their sign, in edge tiles and others."""
    import bit_kv_cache_spc_gb300 as spc
    L = 300
    q, k, v = rnd(1, L, 2, D, mul=0.1), rnd(2, L, 1, D, mul=0.1), rnd(3, L, 1, D)
    v[5, 0, 3], v[130, 0, 7], v[260, 0, 9], v[131, 0, 7], v[290, 0, 11] = math.inf, -math.inf, math.nan, math.inf, -math.inf
    o = torch.zeros_like(q)
    spc.spc_prompt_attn(q, k, v, o)
    assert bool((o[5:, :, 3] == math.inf).all()) and bool(torch.isfinite(o[:5, :, 3]).all())
    assert bool((o[130, :, 7] == -math.inf).all()) and bool(torch.isnan(o[131:, :, 7]).all())
    assert bool(torch.isnan(o[260:, :, 9]).all()) and bool(torch.isfinite(o[:260, :, 9]).all())
    assert bool((o[290:, :, 11] == -math.inf).all()) and bool(torch.isfinite(o[:290, :, 11]).all())
    kept = [c for c in range(D) if c not in (3, 7, 9, 11)]
    vz = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    o2 = torch.zeros_like(q)
    spc.spc_prompt_attn(q, k, vz, o2)
    assert torch.equal(o[:, :, kept], o2[:, :, kept])


@pytest.mark.parametrize("S,most", [(40, 700), (256, 300), (300, 300)])
def test_many_packed_sequences(S, most):
    """Dozens and hundreds of sequences of very different lengths, empty ones among them: every one is done, once."""
    import bit_kv_cache_spc_gb300 as spc
    lens = [(s * 97) % 41 if s % 13 else (most if s == 0 else most // (1 + s % 7)) for s in range(S)]
    begin = [sum(lens[:s]) for s in range(S)]
    T, Hq, Hkv = sum(lens), 2, 1
    q, k, v = rnd(1, T, Hq, D), rnd(2, T, Hkv, D), rnd(3, T, Hkv, D)
    o, lse = torch.full_like(q, 7.0), torch.full((T, Hq), 7.0, device="cuda")
    spc.spc_prompt_attn(q, k, v, o, lse, q_begin=i32(begin), q_len=i32(lens), k_begin=i32(begin), k_len=i32(lens),
                        q_max=most, k_max=most)
    assert not bool((lse == 7).any())
    for s in list(range(0, S, 13)) + [1, 2, S - 1]:
        b, n = begin[s], lens[s]
        if n:
            check(o[b:b + n], lse[b:b + n], q[b:b + n], k[b:b + n], v[b:b + n])


def test_a_large_batch_of_single_tokens():
    """600 sequences of one new token each, packed, over keys that some of them share."""
    import bit_kv_cache_spc_gb300 as spc
    S, T, Hq, Hkv = 600, 900, 4, 1
    q, k, v = rnd(1, S, Hq, D), rnd(2, T, Hkv, D), rnd(3, T, Hkv, D)
    lk = [1 + (s * 53) % 300 for s in range(S)]
    kb = [(s * 31) % 600 for s in range(S)]
    o, lse = torch.zeros_like(q), torch.zeros((S, Hq), device="cuda")
    spc.spc_prompt_attn(q, k, v, o, lse, q_begin=torch.arange(S, dtype=torch.int32, device="cuda"),
                        k_begin=i32(kb), k_len=i32(lk), q_max=1, k_max=300)
    for s in range(0, S, 7):
        check(o[s:s + 1], lse[s:s + 1], q[s:s + 1], k[kb[s]:kb[s] + lk[s]], v[kb[s]:kb[s] + lk[s]])


def test_other_strides_and_scale():
    """Head-major queries and outputs inside wider buffers, and a scale of the caller's."""
    import bit_kv_cache_spc_gb300 as spc
    L, Hq, Hkv = 150, 4, 2
    q = rnd(1, Hq, 2 * L, D)[:, ::2].transpose(0, 1)
    k = rnd(2, L, Hkv, 2, D)[:, :, 1]
    v = rnd(3, Hkv, L, 3 * D)[:, :, D:2 * D].transpose(0, 1)
    ob = torch.full((Hq, L, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    o = ob[:, :, D:].transpose(0, 1)
    spc.spc_prompt_attn(q, k, v, o, scale=0.03)
    check(o, None, q, k, v, scale=0.03)
    assert bool((ob[:, :, :D] == 7).all())


def test_device_lengths_are_held_to_the_tensors():
    """Lengths and first tokens outside the tensors and the stated maxima are cut, and write nothing outside."""
    import bit_kv_cache_spc_gb300 as spc
    T, Hq, Hkv = 100, 4, 2
    q, k, v = rnd(1, T, Hq, D), rnd(2, T, Hkv, D), rnd(3, T, Hkv, D)
    buf = torch.full((T + 300, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    o = buf[150:150 + T]
    spc.spc_prompt_attn(q, k, v, o, q_begin=i32([-5, 90]), q_len=i32([30, 1000]), k_begin=i32([0, 80]),
                        k_len=i32([30, 1 << 30]), q_max=40, k_max=60)
    check(o[:30], None, q[:30], k[:30], v[:30])
    check(o[90:], None, q[90:], k[80:], v[80:])
    assert bool((buf[:150] == 7).all()) and bool((buf[150 + 30:150 + 90] == 7).all()) and bool((buf[150 + T:] == 7).all())


def test_graphs_and_streams_repeat_the_same_bits():
    """Captured and replayed, on another stream, two calls at once with their own workspaces: the same bits."""
    import bit_kv_cache_spc_gb300 as spc
    q, k, v = rnd(1, 1, 32, D), rnd(2, 3000, 8, D), rnd(3, 3000, 8, D)
    o, lse = torch.zeros_like(q), torch.zeros((1, 32), device="cuda")
    need = spc.spc_prompt_attn_workspace_bytes(q, k, v, o)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    assert need > 256  # one query over a long history: the keys are split
    spc.spc_prompt_attn(q, k, v, o, lse, ws=ws)
    want = (o.clone(), lse.clone())
    o.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        spc.spc_prompt_attn(q, k, v, o, lse, ws=ws)
    o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(o) for _ in side]
    wss = [torch.zeros_like(ws) for _ in side]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, x, w in zip(side, outs, wss):
            spc.spc_prompt_attn(q, k, v, x, ws=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[0]) for x in outs)
    assert spc.spc_prompt_attn_status(ws) == 0
