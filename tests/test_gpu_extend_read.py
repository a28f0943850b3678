"""A run of tokens written into the low-bit cache (spc_extend_kv) and the cache read back (spc_dequantize_kv), against
the oracle, bit for bit."""
import numpy as np
import pytest
import torch

import oracle
import synth
from quant_edge import edge_kv

pytestmark = pytest.mark.gpu
D = 128


def dev16(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda()


def levels(mm, code, bits):
    """fl(z + fl(s code)) in binary32, rounded to bf16, of (min, max) patterns broadcast against codes."""
    with np.errstate(all="ignore"):
        lo, hi = (synth.bf16_to_f32(mm[..., i]).astype(np.float32) for i in (0, 1))
        f = np.float32
        if bits == 1:
            z, s = (f(3) * lo + hi) * f(0.25), (hi - lo) * f(0.5)
        else:
            z, s = lo, (hi - lo) / f(3)
        x = z + s * code.astype(np.float32)
        return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)


def expected_rows(od, K, V):
    """bf16 [B][Hkv][N][D] of keys and values that the cache of K, V (bf16 bits) holds."""
    g, nq = od.group, oracle.nq(od)
    qz = oracle.quantize(od, K, V)
    k = torch.from_numpy(K.view(np.int16).copy()).view(torch.bfloat16)
    v = torch.from_numpy(V.view(np.int16).copy()).view(torch.bfloat16)
    if nq:
        k[:, :, :nq] = levels(np.repeat(qz["kmm"], g, axis=2), qz["kcode"], od.bits)
        v[:, :, :nq] = levels(np.repeat(qz["vmm"], g, axis=3), qz["vcode"], od.bits)
    return k, v


def same(a, b):
    """Equal bit for bit, any NaN equal to any."""
    a, b = a.contiguous(), b.contiguous()
    nan = torch.isnan(a)
    return torch.equal(nan, torch.isnan(b)) and torch.equal(a.view(torch.int16)[~nan], b.view(torch.int16)[~nan])


class Cache:
    """An empty cache of room for N tokens, filled by calls."""

    def __init__(self, B, Hkv, N, R, bits, group, host=False):
        import bit_kv_cache_spc_gb300 as spc
        self.spc = spc
        self.od = oracle.dims(B=B, Hq=Hkv, Hkv=Hkv, N=N, R=R, bits=bits, group=group)
        nq = oracle.nq(self.od)
        self.d = spc.Dims(B, Hkv, Hkv, 0, R, bits, q_groups_cap=nq // 32 + 4, resid_cap=R + group + 2, group=group)
        self.rec = torch.full((spc.spc_records_bytes(self.d),), 0xA5, dtype=torch.uint8, device="cuda")
        self.res = torch.full((spc.spc_resid_bytes(self.d) // 2,), 7, dtype=torch.int16, device="cuda")
        self.host = torch.full((B, Hkv, N + 3, 2, D), 7, dtype=torch.int16, pin_memory=True) if host else None

    def extend(self, k, v, stream=None):
        n_cap = 0 if self.host is None else self.host.shape[2]
        self.spc.spc_extend_kv(self.d, k, v, self.rec, self.res, self.host, n_cap, stream=stream)
        self.d.N += k.shape[1]

    def check(self, K, V):
        """The cache holds what the oracle makes of all tokens so far."""
        B, Hkv, N = K.shape[:3]
        K, V = np.ascontiguousarray(K), np.ascontiguousarray(V)
        od = oracle.dims(B=B, Hq=Hkv, Hkv=Hkv, N=N, R=self.od.R, bits=self.od.bits, group=self.od.group)
        nq = oracle.nq(od)
        orec, ores = oracle.pack(od, oracle.quantize(od, K, V), K, V)
        got = self.rec.cpu().numpy().reshape(B, Hkv, oracle.records_per_pair(od.group, self.d.q_groups_cap), -1)
        units = nq // od.group
        assert np.array_equal(got[:, :, :units], orec[:, :, :units]), "records differ"
        assert bool((got[:, :, units:] == 0xA5).all()), "records behind the last one were written"
        res = self.res.cpu().numpy().view(np.uint16).reshape(B, Hkv, self.d.resid_cap, 2, D)
        assert np.array_equal(res[:, :, :N - nq], ores[:, :, :N - nq]), "window differs"
        if self.host is not None:
            h = self.host.numpy().view(np.uint16)
            assert np.array_equal(h[:, :, :N], np.stack([K, V], axis=3)) and bool((h[:, :, N:] == 7).all())


RUNS = [(0, 32, [1]), (0, 32, [300]), (0, 32, [31, 1, 32, 200]), (16, 32, [50, 77, 1, 1, 130]), (128, 32, [100, 29, 400]),
        (200, 32, [700, 5, 64, 33]), (0, 64, [64, 63, 130]), (16, 64, [10, 70, 300]), (130, 64, [129, 66, 500, 2]),
        (5, 32, [36, 31, 33]), (300, 32, [100, 100, 150, 40])]


@pytest.mark.parametrize("bits", [1, 2])
@pytest.mark.parametrize("R,group,runs", RUNS, ids=lambda x: str(x))
def test_runs_match_the_oracle(R, group, runs, bits):
    """Run after run from views of a fused projection, with the offload; the cache and the host rows after each."""
    B, Hkv, N = 2, 3, sum(runs)
    K, V = synth.kv_layer(5, bits, B, Hkv, N)
    c = Cache(B, Hkv, N, R, bits, group, host=True)
    fused = dev16(np.concatenate([K, V], axis=1).transpose(0, 2, 1, 3))  # [B][N][2 Hkv][D]
    at = 0
    for n in runs:
        x = fused[:, at:at + n]
        c.extend(x[:, :, :Hkv], x[:, :, Hkv:])
        torch.cuda.synchronize()
        at += n
        c.check(K[:, :, :at], V[:, :, :at])


@pytest.mark.parametrize("bits,group", [(1, 32), (2, 64)])
def test_runs_of_many_heads_match_the_oracle(bits, group):
    """More (b, KV head) pairs than a single launch takes: old rows move after the groups' own launch."""
    B, Hkv, runs = 13, 8, [150, 20, 70, 1, 200]
    K, V = synth.kv_layer(6, bits, B, Hkv, sum(runs))
    c = Cache(B, Hkv, sum(runs), 70, bits, group, host=True)
    at = 0
    for n in runs:
        k, v = (dev16(np.ascontiguousarray(x[:, :, at:at + n])).transpose(1, 2) for x in (K, V))
        c.extend(k, v)
        torch.cuda.synchronize()
        at += n
    c.check(K, V)


@pytest.mark.parametrize("bits", [1, 2])
@pytest.mark.parametrize("group", [32, 64])
def test_edge_values(bits, group):
    """Groups on the decision boundaries and at the edges of binary32; head-major rows."""
    B, Hkv, N, R = 2, 3, 16 * group + 9, 0
    K, V = edge_kv(3, B, Hkv, N, group=group)
    c = Cache(B, Hkv, N, R, bits, group)
    k, v = dev16(K).transpose(1, 2), dev16(V).transpose(1, 2)
    cut = 3 * group + 5
    c.extend(k[:, :cut], v[:, :cut])
    c.extend(k[:, cut:], v[:, cut:])
    torch.cuda.synchronize()
    c.check(K, V)
    out = torch.empty((2, B, N, Hkv, D), dtype=torch.bfloat16, device="cuda")
    c.spc.spc_dequantize_kv(c.d, c.rec, c.res, 0, out[0], out[1])
    od = oracle.dims(B=B, Hq=Hkv, Hkv=Hkv, N=N, R=R, bits=bits, group=group)
    for got, want in zip(out, expected_rows(od, K, V)):
        assert same(got.cpu().transpose(1, 2), want)


def test_same_as_appends():
    """n tokens at once leave the same bytes as n single appends, from a quantised prompt on."""
    import bit_kv_cache_spc_gb300 as spc
    B, Hkv, N0, n, R = 2, 2, 75, 90, 16
    K, V = synth.kv_layer(6, 0, B, Hkv, N0 + n)
    for bits in (1, 2):
        d = spc.Dims(B, Hkv, Hkv, N0, R, bits, q_groups_cap=8, resid_cap=R + 33)
        kt, vt = dev16(K), dev16(V)
        bufs = []
        for _ in range(2):
            rec = torch.zeros(spc.spc_records_bytes(d), dtype=torch.uint8, device="cuda")
            res = torch.zeros(spc.spc_resid_bytes(d) // 2, dtype=torch.int16, device="cuda")
            spc.spc_quantize_kv(d, kt[:, :, :N0].contiguous(), vt[:, :, :N0].contiguous(), rec, res)
            bufs.append((rec, res))
        spc.spc_extend_kv(d, kt[:, :, N0:].transpose(1, 2), vt[:, :, N0:].transpose(1, 2), *bufs[0])
        d1 = spc.Dims(B, Hkv, Hkv, N0, R, bits, q_groups_cap=8, resid_cap=R + 33)
        for t in range(N0, N0 + n):
            spc.spc_append_kv(d1, kt[:, :, t].contiguous(), vt[:, :, t].contiguous(), *bufs[1])
            d1.N += 1
        r = N0 + n - spc.spc_num_quantized(d1)
        assert torch.equal(bufs[0][0], bufs[1][0])
        x, y = (b[1].view(B, Hkv, -1, 2, D)[:, :, :r] for b in bufs)
        assert torch.equal(x, y)


@pytest.mark.parametrize("bits", [1, 2])
@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("N,R", [(1, 0), (31, 32), (64, 0), (200, 16), (333, 128)])
def test_read_back(N, R, group, bits):
    """Every part of the cache, into views whose other rows keep their bytes."""
    B, Hkv = 2, 3
    K, V = synth.kv_layer(7, bits, B, Hkv, N)
    c = Cache(B, Hkv, N, R, bits, group)
    c.extend(dev16(K).transpose(1, 2), dev16(V).transpose(1, 2))
    od = oracle.dims(B=B, Hq=Hkv, Hkv=Hkv, N=N, R=R, bits=bits, group=group)
    want = expected_rows(od, K, V)
    nq = oracle.nq(od)
    parts = {(0, N), (N - 1, 1), (N // 3, N - N // 3), (min(5, N - 1), 1), (max(nq - 1, 0), min(2, N - max(nq - 1, 0)))}
    for first, n in parts:
        kb = torch.full((B, Hkv, n + 4, D), 7.0, dtype=torch.bfloat16, device="cuda")  # head-major buffer
        vb = torch.full((B, n + 4, Hkv, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
        c.spc.spc_dequantize_kv(c.d, c.rec, c.res, first, kb[:, :, 2:2 + n].transpose(1, 2), vb[:, 2:2 + n, :, D:])
        torch.cuda.synchronize()
        assert same(kb[:, :, 2:2 + n].cpu(), want[0][:, :, first:first + n])
        assert same(vb[:, 2:2 + n, :, D:].cpu().transpose(1, 2), want[1][:, :, first:first + n])
        assert bool((kb[:, :, :2] == 7).all()) and bool((kb[:, :, 2 + n:] == 7).all())
        assert bool((vb[..., :D] == 7).all()) and bool((vb[:, :2] == 7).all()) and bool((vb[:, 2 + n:] == 7).all())


def test_captured_and_on_another_stream():
    """A turn captured with its read-back: each replay works on the rows that the buffers hold then."""
    B, Hkv, N0, n, R, bits, group = 1, 2, 150, 45, 16, 1, 32
    K, V = synth.kv_layer(8, 0, B, Hkv, N0 + n)
    c = Cache(B, Hkv, N0 + n, R, bits, group)
    s = torch.cuda.Stream()
    k, v = dev16(K).transpose(1, 2), dev16(V).transpose(1, 2)
    torch.cuda.synchronize()
    c.extend(k[:, :N0], v[:, :N0], stream=s)
    s.synchronize()
    start = (c.rec.clone(), c.res.clone())
    kn, vn = torch.zeros((2, B, n, Hkv, D), dtype=torch.int16, device="cuda")
    out = torch.zeros((2, B, N0 + n, Hkv, D), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.extend(kn, vn)
        c.spc.spc_dequantize_kv(c.d, c.rec, c.res, 0, out[0], out[1])
    c.rec.copy_(start[0])
    c.res.copy_(start[1])
    kn.copy_(k[:, N0:])
    vn.copy_(v[:, N0:])
    g.replay()
    torch.cuda.synchronize()
    c.check(K, V)
    od = oracle.dims(B=B, Hq=Hkv, Hkv=Hkv, N=N0 + n, R=R, bits=bits, group=group)
    for got, want in zip(out, expected_rows(od, K, V)):
        assert same(got.cpu().transpose(1, 2), want)


@pytest.mark.parametrize("bits,group", [(1, 32), (2, 32), (1, 64), (2, 64)])
def test_prompt_at_a_workload_shape(bits, group):
    """LLaMA-3-8B layer shape (32/8 heads, R = 128), a 32768-token prompt out of a fused projection: the same bytes as
    spc_quantize_kv."""
    import bit_kv_cache_spc_gb300 as spc
    B, Hq, Hkv, N, R = 2, 32, 8, 32768, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    qkv = torch.randn((B, N, Hq + 2 * Hkv, D), generator=g, device="cuda", dtype=torch.bfloat16)
    k, v = qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    d = spc.Dims(B, Hq, Hkv, N, R, bits, group=group)
    rec = torch.zeros((2, spc.spc_records_bytes(d)), dtype=torch.uint8, device="cuda")
    res = torch.zeros((2, spc.spc_resid_bytes(d) // 2), dtype=torch.int16, device="cuda")
    spc.spc_quantize_kv(d, k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous(), rec[0], res[0])
    d0 = spc.Dims(B, Hq, Hkv, 0, R, bits, q_groups_cap=d.q_groups_cap, resid_cap=d.resid_cap, group=group)
    spc.spc_extend_kv(d0, k, v, rec[1], res[1])
    assert torch.equal(rec[0], rec[1]) and torch.equal(res[0], res[1])


@pytest.mark.parametrize("bits,group", [(1, 32), (2, 32), (1, 64), (2, 64)])
def test_non_finite_elements_as_the_quantiser_codes_them(bits, group):
    """Infinities and NaN among the elements: the same records as spc_quantize_kv's."""
    import bit_kv_cache_spc_gb300 as spc
    B, Hkv, N = 2, 2, 8 * group
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    kv = torch.randn((2, B, Hkv, N, D), generator=g, device="cuda").to(torch.bfloat16)
    at = torch.rand((2, B, Hkv, N, D), generator=g, device="cuda")
    for i, x in enumerate((float("nan"), float("inf"), -float("inf"))):
        kv[(at > 0.002 * i) & (at < 0.002 * i + 0.001)] = x
    kv[:, 0, 0, :group] = float("nan")  # groups of nothing else
    kv[:, 0, 1, :group, :64] = float("inf")
    d = spc.Dims(B, Hkv, Hkv, N, 0, bits, group=group)
    rec = torch.zeros((2, spc.spc_records_bytes(d)), dtype=torch.uint8, device="cuda")
    spc.spc_quantize_kv(d, kv[0], kv[1], rec[0], None)
    d0 = spc.Dims(B, Hkv, Hkv, 0, 0, bits, q_groups_cap=d.q_groups_cap, group=group)
    spc.spc_extend_kv(d0, kv[0].transpose(1, 2), kv[1].transpose(1, 2), rec[1], None)
    assert torch.equal(rec[0], rec[1])
