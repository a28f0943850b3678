"""Plain 64-bit form of the prompt attention and its error bounds, for the GPU
tests (torch, on the tensors' device)."""
from __future__ import annotations

import math

import torch

BF16 = 2.0 ** -8   # half a bf16 step, relative to the value
FP32 = 2.0 ** -24  # half a binary32 step


def attention(q, k, v, scale):
    """o, lse and bounds of both for one sequence: q [lq][Hq][D], k, v [lk][Hkv][D] (any 16-bit float).

    The bound of o counts, per element: every weight's rounding to bf16 (half a step of the weight), the store's
    rounding, and the scores' error e in the exponents (128 exact products summed in binary32, at most one
    rounding step, 2^-23, a term of the magnitudes' sum; the multiply-add, at twice the score in powers of two; the
    hardware exponential's 2^-22), which moves each weight and the sum of weights by a factor 1 + e."""
    lq, Hq, D = q.shape
    lk, Hkv = k.shape[0], k.shape[1]
    o = torch.zeros((lq, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((lq, Hq), -math.inf, dtype=torch.float64, device=q.device)
    o_tol, lse_tol = torch.zeros_like(o), torch.zeros_like(lse)
    first = max(lq - lk, 0)  # queries before see nothing
    if lk == 0 or first >= lq:
        return o, lse, o_tol, lse_tol
    seen = torch.ones((lq, lk), dtype=torch.bool, device=q.device).tril(lk - lq)[first:]
    for h in range(Hq):
        qs, ks, vs = q[first:, h].double(), k[:, h * Hkv // Hq].double(), v[:, h * Hkv // Hq].double()
        s = (qs @ ks.T * scale).where(seen, -math.inf)
        z = torch.logsumexp(s, 1)
        p = torch.exp(s - z[:, None])
        mag = (qs.abs() @ ks.abs().T * scale).where(seen, 0.0).amax(1)
        e = 2 * (D * 2 * FP32 * mag + 6 * FP32 * s.where(seen, 0.0).abs().amax(1) + 2.0 ** -21)
        a = p @ vs.abs()
        lse[first:, h], o[first:, h] = z, p @ vs
        o_tol[first:, h] = a * (BF16 * (1 + BF16) + e[:, None] + lk * FP32) + BF16 * (1 + BF16) * o[first:, h].abs() + 1e-30
        lse_tol[first:, h] = e + lk * FP32 + 4 * FP32 * z.abs()
    return o, lse, o_tol, lse_tol
