"""The prompt path of layers with head norms, positions of several axes, sliding windows and shared prefixes, as it is used
(steps.prompt_layer): prompts of a conversation, then a decode step on what they wrote."""
import math

import numpy as np
import pytest
import torch

import oracle
from sight_ref import check, prefix_sight, window_sight
from spc_cases import OUT_TOL, b2f, out_err
from test_gpu_extend_read import expected_rows, same
from test_gpu_norm_rope import check as check_norm

pytestmark = pytest.mark.gpu
D = 128


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class Model:
    """One layer's weights and cache."""

    def __init__(self, B, Hq, Hkv, R, nbits, group, total, axes):
        import bit_kv_cache_spc_gb300 as spc
        self.spc, self.B, self.Hq, self.Hkv, self.total, self.axes = spc, B, Hq, Hkv, total, axes
        self.cap, self.group = total // 32 + 2, group
        self.d = spc.Dims(B, Hq, Hkv, 0, R, nbits, q_groups_cap=self.cap, resid_cap=R + group, group=group)
        self.od = lambda N: oracle.dims(B=B, Hq=Hq, Hkv=Hkv, N=N, R=R, bits=nbits, group=group)
        self.rec = torch.zeros(spc.spc_records_bytes(self.d), dtype=torch.uint8, device="cuda")
        self.res = torch.zeros(spc.spc_resid_bytes(self.d) // 2, dtype=torch.int16, device="cuda")
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(11)
        self.turns = spc.spc_rope_frequencies(64, 10000.0)[0]
        self.axis = spc.spc_rope_axes([12, 10, 10], 64, "turns") if axes == 3 else [0] * 32
        self.wq, self.wk = (1 + 0.3 * torch.randn(D, generator=self.g, device="cuda") for _ in range(2))
        self.K = self.V = None  # every token's normed and rotated key and value row so far, [B][N][Hkv][D]

    def prompt(self, n, B=None):
        B = self.B if B is None else B
        qkv = torch.randn((B, n, self.Hq + 2 * self.Hkv, D), generator=self.g, device="cuda").to(torch.bfloat16)
        q, k, v = qkv[:, :, :self.Hq], qkv[:, :, self.Hq:self.Hq + self.Hkv], qkv[:, :, self.Hq + self.Hkv:]
        t = self.d.N + torch.arange(n, device="cuda", dtype=torch.int32).expand(B, n)
        pos = torch.stack([t, t // 5, t % 7][:self.axes]).contiguous()
        o = torch.full((B, n, self.Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        return q, k, v, pos, o, torch.full((B, n, self.Hq), 7.0, device="cuda")

    def norm(self):
        kw = dict(rot=64, q_norm=self.wq, k_norm=self.wk, eps=1e-5)
        return dict(kw, axis=self.axis) if self.axes > 1 else kw

    def check_rows(self, got, was, w, pos):
        check_norm(got, was, w, 1e-5, pos, self.turns, self.axis, 64, False)

    def history(self, N):
        """The cache's rows as it holds them, [B][N][Hkv][D]."""
        if N == 0:
            return tuple(torch.empty((self.B, 0, self.Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        want = expected_rows(self.od(N), bits(self.K.transpose(1, 2)), bits(self.V.transpose(1, 2)))
        return tuple(x.cuda().transpose(1, 2) for x in want)

    def joined(self, k, v):
        self.K = k.clone() if self.K is None else torch.cat([self.K, k], dim=1)
        self.V = v.clone() if self.V is None else torch.cat([self.V, v], dim=1)

    def check_cache(self):
        """The cache is the oracle's of all tokens, and a decode step attends over it."""
        N = self.d.N
        Kb, Vb, od = bits(self.K.transpose(1, 2)), bits(self.V.transpose(1, 2)), self.od(N)
        qz = oracle.quantize(od, Kb, Vb)
        orec, _ = oracle.pack(od, qz, Kb, Vb)
        units = oracle.nq(od) // self.group
        got = self.rec.cpu().numpy().reshape(self.B, self.Hkv, oracle.records_per_pair(self.group, self.cap), -1)
        assert np.array_equal(got[:, :, :units], orec[:, :, :units])
        q2 = torch.randn((self.B, 2, self.Hq, D), generator=self.g, device="cuda").to(torch.bfloat16)
        o2 = torch.zeros((self.B, 2, self.Hq, D), dtype=torch.int16, device="cuda")
        ws = torch.zeros(self.spc.spc_attn_workspace_bytes(self.d, 0), dtype=torch.uint8, device="cuda")
        self.spc.spc_decode_attn2(self.d, self.rec, self.res, q2, o2, None, None, ws)
        oo, _, _ = oracle.attention(od, bits(q2), qz, Kb, Vb)
        assert out_err(b2f(o2.cpu().numpy()), oo) <= OUT_TOL


@pytest.mark.parametrize("B,Hq,Hkv,R,nbits,group,axes,window,sinks,turns_", [
    (1, 4, 1, 16, 1, 32, 1, 50, 3, [70, 45, 1]), (2, 4, 2, 32, 2, 64, 3, 20, 0, [200, 33, 90, 1]),
    (2, 8, 8, 0, 1, 64, 3, 300, 5, [64, 129, 200]), (1, 8, 2, 128, 1, 32, 1, 1, 1, [100, 90, 300])])
def test_windowed_prompts_with_norms(B, Hq, Hkv, R, nbits, group, axes, window, sinks, turns_):
    """The buffers of the history are full of NaN: what no query sees is neither read back nor used."""
    from bit_kv_cache_spc_gb300.steps import prompt_layer
    total = sum(turns_)
    m = Model(B, Hq, Hkv, R, nbits, group, total, axes)
    side = torch.cuda.Stream()
    for turn, n in enumerate(turns_):
        N = m.d.N
        q, k, v, pos, o, lse = m.prompt(n)
        q0, k0 = q.clone(), k.clone()
        history = torch.full((2, B, Hkv, total + 3, D), math.nan, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        prompt_layer(m.d, q, k, v, pos if axes > 1 else pos[0], m.turns.cuda(), o, m.rec, m.res, history=history, lse=lse,
                     stream=side if turn % 2 else None, window=window, sinks=sinks, **m.norm())
        torch.cuda.synchronize()
        assert m.d.N == N + n
        kr = k if N == 0 else history[0, :, :, N:N + n].transpose(1, 2)
        m.check_rows(q, q0, m.wq, pos)
        m.check_rows(kr, k0, m.wk, pos)
        hk, hv = m.history(N)
        seen = window_sight(n, N + n, window, sinks)
        if N:
            unread = ~seen.any(0)[:N]
            assert bool(torch.isnan(history[:, :, :, :N][:, :, :, unread]).all())
            assert same(history[0, :, :, :N][:, :, ~unread].cpu(), hk.transpose(1, 2)[:, :, ~unread].cpu())
        for b in range(B):
            check(o[b], lse[b], q[b], torch.cat([hk[b], kr[b]]), torch.cat([hv[b], v[b]]), seen)
        m.joined(kr, v)
    m.check_cache()


@pytest.mark.parametrize("B,Hq,Hkv,R,nbits,group,P,turns_", [
    (3, 4, 2, 16, 1, 32, 100, [45, 1, 60]), (5, 8, 2, 32, 2, 64, 333, [1, 1, 7]), (2, 4, 4, 0, 1, 32, 64, [200, 33])])
def test_prompts_behind_a_shared_prefix(B, Hq, Hkv, R, nbits, group, P, turns_):
    """The prefix is a prompt of one sequence; all caches take its rows, and follow-up prompts attend to its 16-bit rows
    once for all and to their own history."""
    from bit_kv_cache_spc_gb300.steps import prompt_layer
    total = P + sum(turns_)
    m = Model(B, Hq, Hkv, R, nbits, group, total, 1)
    q, k, v, pos, o, lse = m.prompt(P, B=1)
    m.spc.spc_norm_rope(q, k, pos[0], m.turns.cuda(), m.wq, m.wk, 1e-5, rot=64)
    pk, pv = k[0], v[0]  # views of the projection
    kp, vp = (x.expand(B, -1, -1, -1).contiguous() for x in (k, v))
    m.spc.spc_extend_kv(m.d, kp, vp, m.rec, m.res)
    m.d.N += P
    m.joined(kp, vp)
    history = torch.full((2, B, Hkv, total - P, D), math.nan, dtype=torch.bfloat16, device="cuda")
    for n in turns_:
        N = m.d.N
        q, k, v, pos, o, lse = m.prompt(n)
        q0, k0 = q.clone(), k.clone()
        prompt_layer(m.d, q, k, v, pos[0], m.turns.cuda(), o, m.rec, m.res, history=history, lse=lse, prefix=(pk, pv), **m.norm())
        assert m.d.N == N + n
        kr = history[0, :, :, N - P:N - P + n].transpose(1, 2)
        m.check_rows(q, q0, m.wq, pos)
        m.check_rows(kr, k0, m.wk, pos)
        hk, hv = m.history(N)
        assert same(history[0, :, :, :N - P].cpu(), hk.transpose(1, 2)[:, :, P:].cpu())
        for b in range(B):
            check(o[b], lse[b], q[b], torch.cat([pk, hk[b, P:], kr[b]]), torch.cat([pv, hv[b, P:], v[b]]), prefix_sight(n, N - P + n, P))
        m.joined(kr, v)
    m.check_cache()


def test_a_captured_layer_behind_a_prefix():
    """Captured and replayed on new projections: the bits of the calls made one by one."""
    from bit_kv_cache_spc_gb300.steps import prompt_layer
    B, Hq, Hkv, P, n = 4, 8, 2, 200, 9
    m = Model(B, Hq, Hkv, 16, 1, 32, P + n, 1)
    _, k, v, _, _, _ = m.prompt(P)
    m.spc.spc_extend_kv(m.d, k, v, m.rec, m.res)
    m.d.N = P
    q, k, v, pos, o, lse = m.prompt(n)
    first = [x.clone() for x in (q, k, v)]
    pk, pv = (torch.randn((P, Hkv, D), generator=m.g, device="cuda").to(torch.bfloat16) for _ in range(2))
    history = torch.zeros((2, B, Hkv, n, D), dtype=torch.bfloat16, device="cuda")
    dev, was = m.turns.cuda(), m.res.clone()

    def layer():
        prompt_layer(m.d, q, k, v, pos[0], dev, o, m.rec, m.res, history=history, lse=lse, prefix=(pk, pv), **m.norm())

    layer()
    want = (o.clone(), lse.clone(), m.res.clone())
    m.d.N = P
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    for x, y in zip((q, k, v), first):
        x.copy_(y)
    m.res.copy_(was)
    o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and torch.equal(m.res, want[2])


def test_refused_layers_change_nothing():
    from bit_kv_cache_spc_gb300 import SpcError
    from bit_kv_cache_spc_gb300.steps import prompt_layer
    B, Hq, Hkv, n = 2, 4, 2, 60
    m = Model(B, Hq, Hkv, 16, 1, 32, 400, 1)
    _, k, v, _, _, _ = m.prompt(100)
    m.spc.spc_extend_kv(m.d, k, v, m.rec, m.res)
    m.d.N = 100
    q, k, v, pos, o, lse = m.prompt(n)
    history = torch.zeros((2, B, Hkv, 170, D), dtype=torch.bfloat16, device="cuda")
    p = torch.zeros((101, Hkv, D), dtype=torch.bfloat16, device="cuda")
    dev = m.turns.cuda()
    state = lambda: [x.clone() for x in (q, k, v, o, lse, m.rec, m.res, history)]  # noqa: E731
    was = state()
    for bad in (dict(window=0), dict(window=5, sinks=-1), dict(prefix=(p, p)), dict(prefix=(p[:50], p[:50]), window=9),
                dict(prefix=(p[:50], p[:40])), dict(prefix=(p[:50, :1], p[:50, :1])), dict(prefix=(p[:50].float(), p[:50].float())),
                dict(history=history[:, :, :, :159]), dict(prefix=(p[:50], p[:50]), history=history[:, :, :, :109]),
                dict(q_norm=m.wq[:64]), dict(k_norm=m.wk, eps=0.0), dict(k_norm=m.wk, eps=math.nan), dict(axis=[1] * 32),
                dict(axis=[0] * 31), dict(prefix=(history[0, 0, :, :50].transpose(0, 1), p[:50]), o=history[0, :, :, :n].transpose(1, 2)),
                dict(window=9, lse=lse[:, :-1].contiguous()), dict(pos=pos)):
        kw = dict(history=history, lse=lse, rot=64)
        kw.update(bad)
        pos_, o_ = kw.pop("pos", pos[0]), kw.pop("o", o)
        if "axis" in bad and bad["axis"] == [1] * 32 or pos_ is pos:
            kw["q_norm"] = m.wq
        if pos_ is pos:
            pos_ = pos.expand(2, -1, -1).contiguous()  # two axes, and no rule for them
        with pytest.raises((ValueError, SpcError)):
            prompt_layer(m.d, q, k, v, pos_, dev, o_, m.rec, m.res, **kw)
        torch.cuda.synchronize()
        assert m.d.N == 100 and all(torch.equal(x, y) for x, y in zip(was, state()))
    prompt_layer(m.d, q, k, v, pos[0], dev, o, m.rec, m.res, history=history, lse=lse, rot=64, prefix=(p[:50], p[:50]))
    assert m.d.N == 160
