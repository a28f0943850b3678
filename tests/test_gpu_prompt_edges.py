"""The prompt path where large calls go: lanes that walk over several heads (spc_rope), single tokens of many sequences
whose keys are split although their CTAs fill the GPU (spc_prompt_attn); and workspaces that are no workspace."""
import math

import pytest
import torch

from prompt_ref import attention
from test_gpu_rope import check as check_rope

pytestmark = pytest.mark.gpu
D = 128


def rnd(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,rot,values,place", [
    (1, 5, 3, 64, True, "out"), (3, 5, 3, 112, True, "out"), (1, 5, 3, 128, False, "in"), (2, 7, 2, 48, True, "in"),
    (1, 0, 5, 64, True, "out"), (1, 6, 0, 96, False, "out")])
@pytest.mark.parametrize("per", [2, 3, 4])
def test_rope_of_lanes_that_walk_over_several_heads(per, B, Hq, Hkv, rot, values, place, inter):
    """Enough rows for `per` heads a lane (one more for each 128 rows an SM), which the heads in all are no multiple of
    in most cases: lanes cross from queries to keys to values, and end early in the last slice.  Every token's rows
    against the 64-bit form."""
    import bit_kv_cache_spc_gb300 as spc
    heads = Hq + Hkv * (2 if values else 1)
    T = -(-(per * 128 * sms() + heads) // (heads * B)) + 3
    turns, m = spc.spc_rope_frequencies(rot, 10000.0, "ramp", 8.0, 1.0, 32.0, 4096.0)
    fused = rnd(per, B, T, Hq + 2 * Hkv, D)
    q = fused[:, :, :Hq] if Hq else None
    k = fused[:, :, Hq:Hq + Hkv] if Hkv else None
    v = fused[:, :, Hq + Hkv:] if values else None
    was = fused.clone()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    pos = torch.randint(0, 1 << 20, (B, T), generator=g, device="cuda", dtype=torch.int32)
    new = lambda x: None if x is None else torch.full((B, x.shape[2], T, D), 7.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)  # noqa: E731
    qo, ko, vo = (new(q), new(k), new(v)) if place == "out" else (None, None, new(v))
    spc.spc_rope(q, k, pos, turns.cuda(), rot=rot, interleaved=inter, mscale=m, v=v, q_out=qo, k_out=ko, v_out=vo)
    if q is not None:
        check_rope(q if qo is None else qo, was[:, :, :Hq], pos, turns, rot, inter, m)
    if k is not None:
        check_rope(k if ko is None else ko, was[:, :, Hq:Hq + Hkv], pos, turns, rot, inter, m)
    if values:
        assert torch.equal(vo, was[:, :, Hq + Hkv:])
    rest = Hq + Hkv if place == "in" else 0
    assert torch.equal(fused[:, :, rest:], was[:, :, rest:])


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("S,Hq,Hkv,most", [(64, 32, 8, 8000), (100, 16, 4, 9000), (77, 8, 8, 12000)])
def test_split_keys_of_sequences_that_fill_the_gpu(S, Hq, Hkv, most, packed):
    """One token each over keys from none to thousands, most of whose splits are empty: every sequence against the
    64-bit form."""
    import bit_kv_cache_spc_gb300 as spc
    lk = [most if s == S // 2 else 0 if s % 9 == 4 else 1 + (s * 977) % 700 if s % 3 else (s * 131) % most for s in range(S)]
    q = rnd(1, S, Hq, D) if packed else rnd(1, S, 1, Hq, D)
    if packed:  # the sequences' keys behind one another
        begin = [sum(lk[:s]) for s in range(S)]
        k, v = rnd(2, sum(lk), Hkv, D), rnd(3, sum(lk), Hkv, D)
        kw = dict(q_begin=torch.arange(S, dtype=torch.int32, device="cuda"), k_begin=i32(begin), q_max=1, k_max=most)
    else:
        kb, vb = rnd(2, S, Hkv, most, D), rnd(3, S, Hkv, most, D)
        k, v, kw = kb.transpose(1, 2), vb.transpose(1, 2), {}
    o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:-1], 7.0, device="cuda")
    assert S * Hkv >= 2 * sms()  # CTAs for all places
    assert spc.spc_prompt_attn_workspace_bytes(q, k, v, o, S=S, q_max=1, k_max=most) > 256
    spc.spc_prompt_attn(q, k, v, o, lse, k_len=i32(lk), **kw)
    for s in range(S):
        n = lk[s]
        kk, vv = (k[begin[s]:begin[s] + n], v[begin[s]:begin[s] + n]) if packed else (k[s, :n], v[s, :n])
        wo, wz, o_tol, z_tol = attention(q[s].view(1, Hq, D), kk, vv, 1 / math.sqrt(D))
        go, gz = o[s].view(1, Hq, D).double(), lse[s].view(1, Hq).double()
        assert bool(((go - wo).abs() <= o_tol).all()), s
        if n:
            assert bool(((gz - wz).abs() <= z_tol).all()), s
        else:
            assert bool((gz == -math.inf).all()), s


def test_a_workspace_that_is_none_is_refused():
    """An expanded tensor's elements are not memory; an address alone says nothing of its size."""
    import bit_kv_cache_spc_gb300 as spc
    q, k, v = rnd(1, 1, 8, D), rnd(2, 4000, 2, D), rnd(3, 4000, 2, D)
    o = torch.full_like(q, 7.0)
    need = spc.spc_prompt_attn_workspace_bytes(q, k, v, o)
    assert need > 256
    room = torch.zeros(2 * need, dtype=torch.uint8, device="cuda")
    for ws in (room[:1].expand(need), room[::2], room.data_ptr(), room.cpu()):
        with pytest.raises(ValueError):
            spc.spc_prompt_attn(q, k, v, o, ws=ws)
    assert bool((o == 7).all())
    spc.spc_prompt_attn(q, k, v, o, ws=room.data_ptr(), ws_bytes=need)
    got = o.clone()
    spc.spc_prompt_attn(q, k, v, o)
    assert torch.equal(got, o)


def test_rows_of_no_elements_are_refused():
    import bit_kv_cache_spc_gb300 as spc
    x = torch.zeros((4, 2, 0), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        spc.spc_prompt_attn(x, x, x, torch.zeros_like(x))


def test_captured_without_a_workspace_of_its_own():
    """Two split calls captured in one graph, each with the workspace it takes: replayed, between other allocations of
    the same sizes, they give the eager calls' bits."""
    import bit_kv_cache_spc_gb300 as spc
    calls = []
    for seed, n in ((1, 4000), (5, 7000)):
        q, k, v = rnd(seed, 1, 8, D), rnd(seed + 1, n, 2, D), rnd(seed + 2, n, 2, D)
        calls.append((q, k, v, torch.zeros_like(q), torch.zeros_like(q)))
    for q, k, v, o, want in calls:
        assert spc.spc_prompt_attn_workspace_bytes(q, k, v, o) > 256
        spc.spc_prompt_attn(q, k, v, want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for q, k, v, o, _ in calls:
            spc.spc_prompt_attn(q, k, v, o)
    for _ in range(3):
        for *_, o, _ in calls:
            o.fill_(7.0)
        other = [torch.full((1 << 18,), math.nan, device="cuda") for _ in range(4)]
        g.replay()
        more = [torch.full((1 << 18,), math.nan, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for *_, o, want in calls)
        del other, more


@pytest.mark.parametrize("before", [0, 300])
def test_a_captured_prompt_layer(before):
    """A prompt's calls captured together (the cache's length is that of the capture): replayed on other projections,
    the bits of the eager call."""
    import bit_kv_cache_spc_gb300 as spc
    from bit_kv_cache_spc_gb300.steps import prompt_layer
    B, n, Hq, Hkv, total = 2, 90, 8, 2, 390
    turns = spc.spc_rope_frequencies(128)[0].cuda()
    made = []
    for captured in (False, True):
        d = spc.Dims(B, Hq, Hkv, 0, 16, 1, q_groups_cap=total // 32 + 1, resid_cap=48)
        rec = torch.zeros(spc.spc_records_bytes(d), dtype=torch.uint8, device="cuda")
        res = torch.zeros(spc.spc_resid_bytes(d) // 2, dtype=torch.int16, device="cuda")
        history = torch.zeros((2, B, Hkv, total, D), dtype=torch.bfloat16, device="cuda")
        o = torch.zeros((B, n, Hq, D), dtype=torch.bfloat16, device="cuda")

        def prompt(x, out):
            at = d.N + torch.arange(x.shape[1], device="cuda", dtype=torch.int32)
            q, k, v = x.split([Hq, Hkv, Hkv], dim=2)
            return lambda: prompt_layer(d, q, k, v, at.expand(B, -1).contiguous(), turns, out, rec, res, history=history)

        if before:
            prompt(rnd(1, B, before, Hq + 2 * Hkv, D), torch.zeros((B, before, Hq, D), dtype=torch.bfloat16, device="cuda"))()
        x = rnd(2, B, n, Hq + 2 * Hkv, D)
        if captured:
            start, empty = (rec.clone(), res.clone()), torch.zeros_like(x)
            call = prompt(empty, o)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call()
            rec.copy_(start[0])
            res.copy_(start[1])
            empty.copy_(x)
            g.replay()
        else:
            prompt(x, o)()
        torch.cuda.synchronize()
        assert d.N == before + n
        made.append((o, rec, res, history))
    assert all(torch.equal(x, y) for x, y in zip(*made))
    assert bool((made[0][0] != 0).any()) and spc.spc_prompt_attn_status() == 0
