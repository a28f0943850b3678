"""The prompt path as it is used (steps.prompt_layer): a prompt, follow-up prompts over the cache read back, then a
decode step on what they wrote."""
import math

import numpy as np
import pytest
import torch

import oracle
from prompt_ref import attention
from spc_cases import OUT_TOL, b2f, out_err
from test_gpu_extend_read import expected_rows, same
from test_gpu_rope import check as check_rope

pytestmark = pytest.mark.gpu
D = 128


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("B,Hq,Hkv,R,nbits,group,turns_", [
    (1, 4, 1, 16, 1, 32, [70, 45, 1]), (2, 4, 2, 32, 2, 64, [200, 33, 90]), (2, 8, 8, 0, 1, 64, [64, 129]),
    (1, 8, 2, 128, 1, 32, [100, 90, 300])])
def test_prompts_of_a_conversation_then_a_decode_step(B, Hq, Hkv, R, nbits, group, turns_):
    import bit_kv_cache_spc_gb300 as spc
    from bit_kv_cache_spc_gb300.steps import prompt_layer
    total = sum(turns_)
    cap = total // 32 + 2
    d = spc.Dims(B, Hq, Hkv, 0, R, nbits, q_groups_cap=cap, resid_cap=R + group, group=group)
    rec = torch.zeros(spc.spc_records_bytes(d), dtype=torch.uint8, device="cuda")
    res = torch.zeros(spc.spc_resid_bytes(d) // 2, dtype=torch.int16, device="cuda")
    host = torch.zeros((B, Hkv, total, 2, D), dtype=torch.int16, pin_memory=True)
    history = torch.zeros((2, B, Hkv, total + 3, D), dtype=torch.bfloat16, device="cuda")
    f, m = spc.spc_rope_frequencies(64, 10000.0, "linear", 2.0)
    side = torch.cuda.Stream()
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    K = V = None  # every token's rotated key and value row so far, [B][N][Hkv][D]
    for turn, n in enumerate(turns_):
        N = d.N
        qkv = torch.randn((B, n, Hq + 2 * Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
        q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        q0, k0 = q.clone(), k.clone()
        pos = (N + torch.arange(n, device="cuda", dtype=torch.int32)).expand(B, n).contiguous()
        o = torch.zeros((B, n, Hq, D), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((B, n, Hq), device="cuda")
        torch.cuda.synchronize()
        prompt_layer(d, q, k, v, pos, f.cuda(), o, rec, res, host, total, history=history, lse=lse, rot=64, mscale=m,
                     stream=side if turn % 2 else None)
        torch.cuda.synchronize()
        assert d.N == N + n
        kr = k if N == 0 else history[0, :, :, N:N + n].transpose(1, 2)
        check_rope(q, q0, pos, f, 64, False, m)
        check_rope(kr, k0, pos, f, 64, False, m)
        if N == 0:
            hk, hv = kr[:, :0], v[:, :0]
        else:  # the history as the cache holds it
            od = oracle.dims(B=B, Hq=Hq, Hkv=Hkv, N=N, R=R, bits=nbits, group=group)
            want = expected_rows(od, bits(K.transpose(1, 2)), bits(V.transpose(1, 2)))
            assert all(same(x[:, :, :N].cpu(), y) for x, y in zip(history, want))
            hk, hv = (x.cuda().transpose(1, 2) for x in want)
        for b in range(B):
            kk, vv = torch.cat([hk[b], kr[b]]), torch.cat([hv[b], v[b]])
            wo, wl, o_tol, l_tol = attention(q[b], kk, vv, 1 / math.sqrt(D))
            assert bool(((o[b].double() - wo).abs() <= o_tol).all())
            assert bool(((lse[b].double() - wl).abs() <= l_tol).all())
        K = kr.clone() if K is None else torch.cat([K, kr], dim=1)
        V = v.clone() if V is None else torch.cat([V, v], dim=1)
    # the cache is the oracle's of all tokens, and a decode step attends over it
    Kb, Vb = bits(K.transpose(1, 2)), bits(V.transpose(1, 2))
    od = oracle.dims(B=B, Hq=Hq, Hkv=Hkv, N=total, R=R, bits=nbits, group=group)
    qz = oracle.quantize(od, Kb, Vb)
    orec, _ = oracle.pack(od, qz, Kb, Vb)
    units = oracle.nq(od) // group
    got = rec.cpu().numpy().reshape(B, Hkv, oracle.records_per_pair(group, cap), -1)
    assert np.array_equal(got[:, :, :units], orec[:, :, :units])
    assert np.array_equal(host.numpy().view(np.uint16), np.stack([Kb, Vb], axis=3))
    q2 = torch.randn((B, 2, Hq, D), generator=g, device="cuda").to(torch.bfloat16)
    o2 = torch.zeros((B, 2, Hq, D), dtype=torch.int16, device="cuda")
    ws = torch.zeros(spc.spc_attn_workspace_bytes(d, 0), dtype=torch.uint8, device="cuda")
    spc.spc_decode_attn2(d, rec, res, q2, o2, None, None, ws)
    oo, _, _ = oracle.attention(od, bits(q2), qz, Kb, Vb)
    assert out_err(b2f(o2.cpu().numpy()), oo) <= OUT_TOL


def test_follow_up_without_room_is_refused():
    import bit_kv_cache_spc_gb300 as spc
    from bit_kv_cache_spc_gb300.steps import prompt_layer
    d = spc.Dims(1, 2, 1, 40, 0, 1, q_groups_cap=4, resid_cap=64)
    x = torch.zeros((1, 5, 2, D), dtype=torch.bfloat16, device="cuda")
    short = torch.zeros((2, 1, 1, 44, D), dtype=torch.bfloat16, device="cuda")
    for history in (None, short):
        with pytest.raises(ValueError):
            prompt_layer(d, x, x[:, :, :1], x[:, :, 1:], None, None, x, None, None, history=history)
    assert d.N == 40
