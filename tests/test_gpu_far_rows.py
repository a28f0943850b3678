"""Rows whose places pass 32 bits: the calls on views with tokens 32 MB apart give the bits of the same calls on dense tensors."""
import math

import pytest
import torch

from sight_ref import i32, rnd

pytestmark = pytest.mark.gpu
D, STEP = 128, 1 << 24  # elements from token to token: more than 2^32 bytes from token 128 on, 2^31 elements


@pytest.fixture(scope="module")
def far():
    """far(name, x): x's rows in a buffer of their own, tokens STEP apart (the last three axes are token, head, D)."""
    buffers = {}

    def place(name, x):
        S, T = (x.shape[0] if x.dim() == 4 else 1), x.shape[-3]
        if name not in buffers:
            buffers[name] = torch.empty(200 * STEP, dtype=torch.bfloat16, device="cuda")
        h = x.shape[-2]
        assert S * h * D <= STEP and T <= 200
        shape = x.shape
        stride = (h * D, STEP, D, 1) if x.dim() == 4 else (STEP, D, 1)
        y = buffers[name].as_strided(shape, stride)
        y.copy_(x)
        return y

    yield place
    buffers.clear()
    torch.cuda.empty_cache()


def both(far, run, **x):
    """The outputs of run(place): on dense tensors, and on far ones."""
    got = []
    for place in (lambda name, t: t, far):
        got.append([t.clone() for t in run(**{n: place(n, t) for n, t in x.items()})])
    assert all(torch.equal(a, b) or torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(*got))


@pytest.mark.parametrize("inter", [False, True])
def test_norms_and_rotation(far, inter):
    import bit_kv_cache_spc_gb300 as spc
    turns = spc.spc_rope_frequencies(128)[0].cuda()
    w, pos = 1 + rnd(9, D).float().abs(), torch.arange(199, dtype=torch.int32, device="cuda")[None]
    q, k, v = rnd(1, 1, 199, 4, D), rnd(2, 1, 199, 2, D), rnd(3, 1, 199, 2, D)

    def run(q, k, v, o, pk, pv):
        spc.spc_norm_rope(q, k, pos, turns, w, w, interleaved=inter, v=v, q_out=o, k_out=pk, v_out=pv)
        return o, pk, pv

    both(far, run, q=q, k=k, v=v, o=torch.zeros_like(q), pk=torch.zeros_like(k), pv=torch.zeros_like(v))


@pytest.mark.parametrize("S,lq,Hq,Hkv", [(1, 1, 8, 2), (3, 1, 8, 2), (1, 40, 8, 2), (2, 190, 4, 1), (16, 190, 24, 24)])
@pytest.mark.parametrize("window,sinks", [(30, 3), (150, 0)])
def test_windows(far, S, lq, Hq, Hkv, window, sinks):
    """Single tokens, few and many tiles (CTAs that stay), an infinity and a NaN among the last values."""
    import bit_kv_cache_spc_gb300 as spc
    q, k, v = rnd(1, S, lq, Hq, D), rnd(2, S, 199, Hkv, D), rnd(3, S, 199, Hkv, D)
    v[:, 190, :, 7], v[:, 195, :, 9] = math.inf, math.nan
    lse = torch.zeros((S, lq, Hq), device="cuda")

    def run(q, k, v, o):
        lse.fill_(7)
        spc.spc_window_attn(q, k, v, o, window, sinks, lse)
        return o, lse

    both(far, run, q=q, k=k, v=v, o=torch.zeros_like(q))


@pytest.mark.parametrize("S,lq,Hq,Hkv,plan", [(1, 1, 8, 2, 1), (5, 1, 8, 2, 1), (64, 7, 16, 4, 0), (1, 190, 8, 2, 0), (70, 2, 16, 4, 0)])
def test_prefixes(far, S, lq, Hq, Hkv, plan):
    import bit_kv_cache_spc_gb300 as spc
    q, k, v = rnd(1, S, lq, Hq, D), rnd(2, S, 195, Hkv, D), rnd(3, S, 195, Hkv, D)
    pk, pv = rnd(4, 199, Hkv, D), rnd(5, 199, Hkv, D)
    v[:, 194, :, 7], pv[198, :, 9] = math.inf, math.nan
    lse = torch.zeros((S, lq, Hq), device="cuda")

    def run(q, k, v, o, pk, pv):
        assert spc.spc_prefix_attn_together(q, pk, pv, k, v, o) == plan
        lse.fill_(7)
        spc.spc_prefix_attn(q, pk, pv, k, v, o, lse)
        return o, lse

    both(far, run, q=q, k=k, v=v, o=torch.zeros_like(q), pk=pk, pv=pv)


@pytest.mark.parametrize("S,Hq,Hkv,m,plan", [(64, 8, 2, 90, 2), (70, 16, 4, 64, 1)])
def test_rows_of_several_sequences(far, S, Hq, Hkv, m, plan):
    """Packed, two tokens each up to the axis's end, own keys anywhere; the prefix is dense."""
    import bit_kv_cache_spc_gb300 as spc
    T, n = 199, 2
    q, k, v, pk, pv = rnd(1, T, Hq, D), rnd(2, T, Hkv, D), rnd(3, T, Hkv, D), rnd(4, 8001, Hkv, D), rnd(5, 8001, Hkv, D)
    v[T - 1, :, 7] = math.inf
    at = dict(q_begin=i32([T - n * (S - s) for s in range(S)]), k_begin=i32([T - m - (s * 31) % (T - m) for s in range(S)]))
    lse = torch.zeros((T, Hq), device="cuda")

    def run(q, k, v, o):
        assert spc.spc_prefix_attn_together(q, pk, pv, k, v, o, S=S, q_max=n, k_max=m, placed=True) == plan
        o.fill_(7)
        lse.fill_(7)
        spc.spc_prefix_attn(q, pk, pv, k, v, o, lse, q_max=n, q_len=i32([n] * S), k_len=i32([m] * S), k_max=m, **at)
        return o, lse

    both(far, run, q=q, k=k, v=v, o=torch.zeros_like(q))
