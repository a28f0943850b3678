"""Head norms with the rotation in the same pass (spc_norm_rope) against a plain 64-bit form."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
D = 128
BF16, FP32 = 2.0 ** -8, 2.0 ** -24


def rnd(seed, *shape, mul=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * mul).to(torch.bfloat16)


def weight(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return 1 + 0.3 * torch.randn(D, generator=g, device="cuda")


def angles(pos, turns, axis):
    """[B][T][pairs] radians of positions [axes][B][T], exact fractions of a turn."""
    rows = [[((int(p) * int(turns[i])) % (1 << 64)) * 2.0 ** -64 for p in pos[a].flatten().tolist()] for i, a in enumerate(axis)]
    a = torch.tensor(rows, dtype=torch.float64, device=pos.device) * (2 * math.pi)
    return a.T.reshape(*pos.shape[1:], len(axis))


def exact(x, w, eps, pos, turns, axis, rot, inter, m=1.0):
    """Value and bound.  The norm: 16 squares a lane and three joins of lanes in binary32 (19 roundings of the sum, which
    move the root's reciprocal by half), eps added (1), the reciprocal root (2 units: 4 half steps), two products: 17 half
    steps.  The rotation: cosine and sine off by a few units of binary32, the angle by 2^-32 turns and its rounding to
    binary32, products and sums.  Then one rounding of the result to bf16."""
    y = x.double()
    rel = 0.0
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * w.double()
        rel = 17 * FP32 * (1 + 1e-5)
    a = angles(pos, turns.tolist(), axis).unsqueeze(2)
    c, s = a.cos() * m, a.sin() * m
    i = torch.arange(rot // 2, device=x.device)
    i0, i1 = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    z, tol = y.clone(), rel * y.abs()
    u, v = y[..., i0], y[..., i1]
    z[..., i0], z[..., i1] = u * c - v * s, u * s + v * c
    mag = (u.abs() + v.abs()) * abs(m) * (rel + 8 * FP32 + math.pi * FP32 + 2 * math.pi * 2.0 ** -32)
    tol[..., i0], tol[..., i1] = mag, mag
    if w is None:
        tol[..., :rot] += BF16 * (z[..., :rot].abs() + tol[..., :rot])
    else:
        tol += BF16 * (z.abs() + tol)
    return z, tol


def check(got, *args, **kw):
    z, tol = exact(*args, **kw)
    err = (got.double() - z).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [16, 48, 64, 112, 128])
@pytest.mark.parametrize("B,T,Hq,Hkv,axes", [(1, 1, 1, 1, 1), (2, 3, 4, 2, 3), (3, 67, 5, 1, 2), (1, 33, 7, 3, 4)])
def test_layouts_parts_and_axes(inter, rot, B, T, Hq, Hkv, axes):
    import bit_kv_cache_spc_gb300 as spc
    turns, m = spc.spc_rope_frequencies(rot, 10000.0, "ramp", 8.0, 1.0, 32.0, 4096.0)
    q, k, v = rnd(1, B, T, Hq, D), rnd(2, B, T, Hkv, D, mul=30.0), rnd(3, B, T, Hkv, D)
    pos = torch.randint(0, 1 << 20, (axes, B, T), device="cuda", dtype=torch.int32)
    axis = [(5 * i + i // 3) % axes for i in range(rot // 2)]
    wq, wk = weight(4), weight(5)
    qo, ko, vo = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    spc.spc_norm_rope(q, k, pos, turns.cuda(), wq, wk, 1e-5, axis, rot, inter, m, v, qo, ko, vo)
    check(qo, q, wq, 1e-5, pos, turns, axis, rot, inter, m)
    check(ko, k, wk, 1e-5, pos, turns, axis, rot, inter, m)
    assert torch.equal(vo, v)


@pytest.mark.parametrize("which", ["q", "k", "none"])
@pytest.mark.parametrize("T", [3, 1500])
def test_norms_of_one_kind_only(which, T):
    """Rows without a weight are rotated as spc_rope does it, bit for bit; also in place in a fused projection."""
    import bit_kv_cache_spc_gb300 as spc
    B, Hq, Hkv, rot = 2, 8, 2, 64
    turns = spc.spc_rope_frequencies(rot)[0]
    dev = turns.cuda()
    qkv = rnd(4, B, T, Hq + 2 * Hkv, D)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    pos = (7 + torch.arange(T, device="cuda", dtype=torch.int32)).expand(B, T).contiguous()
    w = weight(9)
    qr, kr = torch.empty_like(q), torch.empty_like(k)
    spc.spc_rope(q, k, pos, dev, rot, q_out=qr, k_out=kr)
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    spc.spc_norm_rope(q, k, pos, dev, w if which == "q" else None, w if which == "k" else None, rot=rot)
    axis = [0] * (rot // 2)
    for name, got, was, rotated in (("q", q, q0, qr), ("k", k, k0, kr)):
        if which == name:
            check(got[:, -5:], was[:, -5:], w, 1e-6, pos[None, :, -5:], turns, axis, rot, False)
        else:
            assert torch.equal(got, rotated)
    assert torch.equal(v, v0)


def test_only_queries_or_only_keys():
    import bit_kv_cache_spc_gb300 as spc
    turns = spc.spc_rope_frequencies(128)[0]
    x, w = rnd(1, 2, 9, 3, D), weight(2)
    pos = torch.arange(18, dtype=torch.int32, device="cuda").view(2, 9)
    a, b = torch.empty_like(x), torch.empty_like(x)
    spc.spc_norm_rope(x, None, pos, turns.cuda(), q_weight=w, q_out=a)
    spc.spc_norm_rope(None, x, pos, turns.cuda(), k_weight=w, k_out=b)
    check(a, x, w, 1e-6, pos[None], turns, [0] * 64, 128, False)
    assert torch.equal(a, b)


@pytest.mark.parametrize("size", [0.0, 1e-30, 1e-3, 1e15, 2.0 ** 62, 1e30, 3e38])
def test_rows_of_any_size(size):
    """From rows of zeros to rows whose squares overflow binary32.  (Below 1e-19 squares are lost beside eps.)"""
    import bit_kv_cache_spc_gb300 as spc
    turns = spc.spc_rope_frequencies(128)[0]
    q = (rnd(1, 1, 5, 2, D).clamp(-1, 1) * size).to(torch.bfloat16)
    w, pos = weight(2), torch.arange(5, dtype=torch.int32, device="cuda")[None]
    out = torch.empty_like(q)
    spc.spc_norm_rope(q, None, pos, turns.cuda(), q_weight=w, q_out=out)
    check(out, q, w, 1e-6, pos[None], turns, [0] * 64, 128, False)


def test_non_finite_elements_stay_in_their_row():
    import bit_kv_cache_spc_gb300 as spc
    turns = spc.spc_rope_frequencies(128)[0]
    q = rnd(1, 1, 40, 3, D)
    clean = torch.empty_like(q)
    pos, w = torch.arange(40, dtype=torch.int32, device="cuda")[None], weight(2)
    spc.spc_norm_rope(q, None, pos, turns.cuda(), q_weight=w, q_out=clean)
    q[0, 1, 0, 3], q[0, 7, 2, 70] = math.nan, math.inf
    out = torch.empty_like(q)
    spc.spc_norm_rope(q, None, pos, turns.cuda(), q_weight=w, q_out=out)
    other = torch.ones((40, 3), dtype=torch.bool, device="cuda")
    other[1, 0] = other[7, 2] = False
    assert torch.equal(out[0][other], clean[0][other])
    assert bool(torch.isnan(out[0, 1, 0]).all())
    inf = out[0, 7, 2]  # an infinite mean: the infinity is no number, in its pair; the others are 0
    assert bool(torch.isnan(inf[[6, 70]]).all()) and bool((inf[[i for i in range(D) if i not in (6, 70)]] == 0).all())


@pytest.mark.parametrize("start", [0, 131071, (1 << 31) - 40, -(1 << 31)])
def test_far_and_negative_positions(start):
    import bit_kv_cache_spc_gb300 as spc
    turns = spc.spc_rope_frequencies(128, 500000.0)[0]
    q, w = rnd(1, 1, 33, 2, D), weight(3)
    t = torch.arange(33, device="cuda", dtype=torch.int64)
    pos = torch.stack([start + t, (start + 7 * t) % (1 << 31), t]).to(torch.int32).view(3, 1, 33)
    axis = spc.spc_rope_axes([24, 20, 20], 128, "turns")
    out = torch.empty_like(q)
    spc.spc_norm_rope(q, None, pos, turns.cuda(), w, axis=axis, q_out=out)
    check(out, q, w, 1e-6, pos, turns, axis, 128, False)


def test_a_long_prompt_into_cache_rows():
    """Many tokens (several heads a group of lanes), rows of the cache around them left as they were."""
    import bit_kv_cache_spc_gb300 as spc
    B, T, Hq, Hkv, cap = 2, 3001, 12, 4, 3010
    turns = spc.spc_rope_frequencies(128)[0]
    qkv = rnd(4, B, T, Hq + 2 * Hkv, D)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    pos = torch.arange(T, device="cuda", dtype=torch.int32).expand(B, T).contiguous()
    kb = torch.full((2, B, Hkv, cap, D), 7.0, dtype=torch.bfloat16, device="cuda")
    kr, vr = (x[:, :, 3:3 + T].transpose(1, 2) for x in kb)
    qo, wq, wk = torch.empty_like(q), weight(1), weight(2)
    spc.spc_norm_rope(q, k, pos, turns.cuda(), wq, wk, v=v, q_out=qo, k_out=kr, v_out=vr)
    for at in (slice(0, 40), slice(1490, 1520), slice(T - 33, T)):
        check(qo[:, at], q[:, at], wq, 1e-6, pos[None, :, at], turns, [0] * 64, 128, False)
        check(kr[:, at], k[:, at], wk, 1e-6, pos[None, :, at], turns, [0] * 64, 128, False)
    assert torch.equal(vr, v)
    assert bool((kb[:, :, :, :3] == 7).all()) and bool((kb[:, :, :, 3 + T:] == 7).all())


def test_captured_and_replayed():
    """New rows, positions and weights are read at replay; on another stream too the same bits."""
    import bit_kv_cache_spc_gb300 as spc
    turns = spc.spc_rope_frequencies(128)[0].cuda()
    q, k, w = rnd(1, 2, 2, 8, D), rnd(2, 2, 2, 2, D), weight(3)
    pos = torch.tensor([[7, 8], [90, 91]], dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        spc.spc_norm_rope(q, k, pos, turns, w, w, q_out=qo, k_out=ko)
    pos += 5
    q.mul_(0.5)
    w.mul_(1.5)
    g.replay()
    torch.cuda.synchronize()
    check(qo, q, w, 1e-6, pos[None], turns.cpu(), [0] * 64, 128, False)
    check(ko, k, w, 1e-6, pos[None], turns.cpu(), [0] * 64, 128, False)
    side, again = torch.cuda.Stream(), torch.empty_like(q)
    spc.spc_norm_rope(q, None, pos, turns, w, q_out=again, stream=side)
    side.synchronize()
    assert torch.equal(again, qo)
