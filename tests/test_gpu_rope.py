"""Rotary positions (spc_rope) against a plain 64-bit form."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
D = 128
BF16 = 2.0 ** -8


def rnd(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def exact(x, pos, turns, rot, inter, m):
    """Value and bound: one rounding of the result; cosine and sine off by a few units of binary32 and the angle by
    2^-32 turns and its rounding to binary32 (2^-24 of at most pi); products and sums of binary32."""
    a = torch.tensor([[((int(p) * int(t)) % (1 << 64)) * 2.0 ** -64 for t in turns.tolist()]
                      for p in pos.flatten().tolist()], dtype=torch.float64, device=x.device)
    a = (a * 2 * math.pi).view(*pos.shape, 1, rot // 2)
    c, s = a.cos() * m, a.sin() * m
    xd = x.double()
    i = torch.arange(rot // 2, device=x.device)
    i0, i1 = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    y, tol = xd.clone(), torch.zeros_like(xd)
    u, w = xd[..., i0], xd[..., i1]
    y[..., i0], y[..., i1] = u * c - w * s, u * s + w * c
    mag = (u.abs() + w.abs()) * abs(m) * (8 * 2.0 ** -24 + math.pi * 2.0 ** -24 + 2 * math.pi * 2.0 ** -32)
    tol[..., i0], tol[..., i1] = mag, mag
    tol[..., :rot] += BF16 * (y[..., :rot].abs() + tol[..., :rot])
    return y, tol


def check(got, x, pos, turns, rot, inter, m):
    y, tol = exact(x, pos, turns, rot, inter, m)
    err = (got.double() - y).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [16, 48, 64, 112, 128])
@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 1, 1), (2, 3, 4, 2), (3, 67, 5, 1)])
def test_layouts_and_parts(inter, rot, B, T, Hq, Hkv):
    import bit_kv_cache_spc_gb300 as spc
    turns, m = spc.spc_rope_frequencies(rot, 10000.0, "ramp", 8.0, 1.0, 32.0, 4096.0)
    q, k, v = rnd(1, B, T, Hq, D), rnd(2, B, T, Hkv, D), rnd(3, B, T, Hkv, D)
    pos = torch.randint(0, 1 << 20, (B, T), device="cuda", dtype=torch.int32)
    qo, ko, vo = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    spc.spc_rope(q, k, pos, turns.cuda(), rot=rot, interleaved=inter, mscale=m, v=v, q_out=qo, k_out=ko, v_out=vo)
    check(qo, q, pos, turns, rot, inter, m)
    check(ko, k, pos, turns, rot, inter, m)
    assert torch.equal(vo, v) and torch.equal(qo[..., rot:], q[..., rot:])


@pytest.mark.parametrize("start", [0, 131071, (1 << 31) - 40, -(1 << 31)])
def test_far_and_negative_positions(start):
    """Angles are exact at any position that an int32 holds."""
    import bit_kv_cache_spc_gb300 as spc
    turns, m = spc.spc_rope_frequencies(128, 500000.0)
    q = rnd(1, 1, 33, 2, D)
    pos = (torch.arange(33, device="cuda", dtype=torch.int64) + start).to(torch.int32)
    out = torch.empty_like(q)
    spc.spc_rope(q, None, pos, turns.cuda(), q_out=out)
    check(out, q, pos.view(1, 33), turns, 128, False, m)


@pytest.mark.parametrize("T", [5, 2000])
def test_in_place_and_out_of_a_fused_projection(T):
    """In place in the fused projection, and from it to head-major cache rows: the same rows; the values' and the
    buffer's other bytes stay."""
    import bit_kv_cache_spc_gb300 as spc
    B, Hq, Hkv, cap = 2, 8, 2, T + 7
    turns, m = spc.spc_rope_frequencies(64, 10000.0, "linear", 2.0)
    dturns = turns.cuda()
    qkv = rnd(4, B, T, Hq + 2 * Hkv, D)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    pos = torch.arange(T, device="cuda", dtype=torch.int32).expand(B, T).contiguous()
    kb = torch.full((2, B, Hkv, cap, D), 7.0, dtype=torch.bfloat16, device="cuda")
    qo = torch.empty_like(q)
    spc.spc_rope(q, k, pos, dturns, rot=64, v=v, q_out=qo, k_out=kb[0, :, :, 3:3 + T].transpose(1, 2),
                 v_out=kb[1, :, :, 3:3 + T].transpose(1, 2))
    v0 = v.clone()
    check(qo[:, -5:], q[:, -5:], pos[:, -5:], turns, 64, False, m)
    spc.spc_rope(q, k, pos, dturns, rot=64)
    assert torch.equal(q, qo) and torch.equal(k, kb[0, :, :, 3:3 + T].transpose(1, 2)) and torch.equal(v, v0)
    assert torch.equal(kb[1, :, :, 3:3 + T].transpose(1, 2), v0)
    assert bool((kb[:, :, :, :3] == 7).all()) and bool((kb[:, :, :, 3 + T:] == 7).all())


def test_turning_back():
    """Position p then -p gives the row back within the two roundings."""
    import bit_kv_cache_spc_gb300 as spc
    turns, _ = spc.spc_rope_frequencies(128, 10000.0)
    q = rnd(1, 1, 64, 3, D)
    pos = torch.arange(1000, 1064, device="cuda", dtype=torch.int32)
    x = q.clone()
    spc.spc_rope(x, None, pos, turns.cuda())
    spc.spc_rope(x, None, -pos, turns.cuda())
    r = torch.hypot(q[..., :64].double(), q[..., 64:].double()).repeat(1, 1, 1, 2)
    # the first rounding moves the pair by at most half a step of its length, turned back with it; then the second
    assert bool(((x.double() - q.double()).abs() <= (2 * BF16 + BF16 ** 2 + 1e-5) * r).all())


def test_non_finite_elements_stay_in_their_pair():
    import bit_kv_cache_spc_gb300 as spc
    turns, _ = spc.spc_rope_frequencies(128, 10000.0)
    q = rnd(1, 1, 4, 2, D)
    q[0, 1, 0, 3], q[0, 2, 1, 70] = math.nan, math.inf
    out = torch.empty_like(q)
    spc.spc_rope(q, None, torch.tensor([1, 2, 3, 4], dtype=torch.int32, device="cuda"), turns.cuda(), q_out=out)
    want = torch.zeros_like(out, dtype=torch.bool)
    want[0, 1, 0, 3] = want[0, 1, 0, 67] = want[0, 2, 1, 6] = want[0, 2, 1, 70] = True
    assert torch.equal(~torch.isfinite(out), want)


def test_captured_and_replayed():
    import bit_kv_cache_spc_gb300 as spc
    turns, _ = spc.spc_rope_frequencies(128, 10000.0)
    dturns = turns.cuda()
    q, k = rnd(1, 2, 2, 8, D), rnd(2, 2, 2, 2, D)
    pos = torch.tensor([[7, 8], [90, 91]], dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        spc.spc_rope(q, k, pos, dturns, q_out=qo, k_out=ko)
    pos += 5  # the step's positions are read at replay
    g.replay()
    torch.cuda.synchronize()
    check(qo, q, pos, turns, 128, False, 1.0)
    check(ko, k, pos, turns, 128, False, 1.0)
