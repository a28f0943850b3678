"""Plain 64-bit form of an attention whose queries each see a set of keys, and its error bounds, for the GPU tests (torch, on
the tensors' device)."""
from __future__ import annotations

import math

import torch

BF16 = 2.0 ** -8   # half a bf16 step, relative to the value
FP32 = 2.0 ** -24  # half a binary32 step
D = 128


def rnd(seed, *shape, mul=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * mul).to(torch.bfloat16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def window_sight(lq, lk, window, sinks):
    """seen [lq][lk]: the last `window` keys up to the query's own place and the first `sinks`."""
    p = torch.arange(lq, device="cuda")[:, None] + (lk - lq)
    j = torch.arange(lk, device="cuda")[None, :]
    return (j <= p) & ((j > p - window) | (j < sinks))


def prefix_sight(lq, lk, P):
    """seen [lq][P + lk]: the prefix, and the sequence's keys that are not behind the query."""
    own = torch.ones((lq, lk), dtype=torch.bool, device="cuda").tril(lk - lq)
    return torch.cat([torch.ones((lq, P), dtype=torch.bool, device="cuda"), own], dim=1)


def attention(q, k, v, seen, scale=D ** -0.5):
    """o, lse and bounds of both for one sequence: q [lq][Hq][D], k, v [lk][Hkv][D] (any 16-bit float), seen [lq][lk].
    What stands in keys and values that a query does not see is not used.

    The bound of o counts, per element: every weight's rounding to bf16 (half a step of the weight), the store's
    rounding, and the scores' error e in the exponents (128 exact products summed in binary32, at most one
    rounding step, 2^-23, a term of the magnitudes' sum; the multiply-add, at twice the score in powers of two; the
    hardware exponential's 2^-22), which moves each weight and the sum of weights by a factor 1 + e.  Parts of the
    keys that are joined afterwards weigh by two more exponentials: counted in e's 2^-20."""
    lq, Hq, _ = q.shape
    lk, Hkv = k.shape[0], k.shape[1]
    o = torch.zeros((lq, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((lq, Hq), -math.inf, dtype=torch.float64, device=q.device)
    o_tol, lse_tol = torch.zeros_like(o), torch.zeros_like(lse)
    rows = seen.any(1)
    if lk == 0 or not bool(rows.any()):
        return o, lse, o_tol, lse_tol
    m = seen[rows]
    for h in range(Hq):
        qs, ks, vs = q[rows, h].double(), k[:, h * Hkv // Hq].double(), v[:, h * Hkv // Hq].double()
        s = (qs @ ks.T * scale).where(m, -math.inf)
        z = torch.logsumexp(s, 1)
        p = torch.exp(s - z[:, None])
        mag = (qs.abs() @ ks.abs().T * scale).where(m, 0.0).amax(1)
        e = 2 * (D * 2 * FP32 * mag + 6 * FP32 * s.where(m, 0.0).abs().amax(1) + 2.0 ** -20)
        a = p @ vs.abs()
        y = p @ vs
        lse[rows, h], o[rows, h] = z, y
        o_tol[rows, h] = a * (BF16 * (1 + BF16) + e[:, None] + lk * FP32) + BF16 * (1 + BF16) * y.abs() + 1e-30
        lse_tol[rows, h] = e + lk * FP32 + 4 * FP32 * z.abs()
    return o, lse, o_tol, lse_tol


def check(got_o, got_lse, q, k, v, seen, scale=D ** -0.5):
    """One sequence's output rows against the 64-bit form."""
    o, lse, o_tol, lse_tol = attention(q, k, v, seen, scale)
    err = (got_o.double() - o).abs()
    assert bool((err <= o_tol).all()), f"o off by {float((err - o_tol).max())} beyond the bound"
    if got_lse is not None:
        none = torch.isinf(lse)
        assert torch.equal(torch.isinf(got_lse) & (got_lse < 0), none)
        err = (got_lse.double() - lse)[~none].abs()
        assert bool((err <= lse_tol[~none]).all()), f"lse off by {float((err - lse_tol[~none]).max())} beyond the bound"
