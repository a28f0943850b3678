"""spc_prefix_attn where tiles hold rows of several sequences: every way in which the prefix's walk and the sequences' own keys
are joined, by shapes that are planned so (asked for and asserted), against a plain 64-bit form."""
import math

import pytest
import torch

from sight_ref import check, i32, prefix_sight, rnd

pytestmark = pytest.mark.gpu
D = 128

# S sequences of up to n queries and m own keys, P shared tokens; plan: own keys in the prefix's walk (2) or in a launch of
# their own (1); joined: the walk's splits through memory, or on the chip.
SHAPES = {
    "packed, in the walk": dict(S=40, n=7, Hq=4, Hkv=2, P=4001, m=7, batched=False, plan=2, joined="memory"),
    "packed, in the walk, on the chip": dict(S=64, n=7, Hq=16, Hkv=4, P=2000, m=7, batched=False, plan=2, joined="chip"),
    "packed, a tile of 42 tokens": dict(S=50, n=9, Hq=6, Hkv=2, P=6001, m=30, batched=False, plan=2, joined="memory"),
    "packed, a shorter last split": dict(S=17, n=77, Hq=16, Hkv=16, P=8011, m=77, batched=False, plan=2, joined="memory"),
    "packed, a token of 32 heads": dict(S=64, n=1, Hq=32, Hkv=1, P=9000, m=20, batched=False, plan=2, joined="memory"),
    "packed, a tile of two tokens": dict(S=50, n=5, Hq=64, Hkv=1, P=9000, m=20, batched=False, plan=2, joined="chip"),
    "packed, apart": dict(S=65, n=7, Hq=8, Hkv=2, P=8001, m=33, batched=False, plan=1, joined="memory"),
    "packed, several hundred, apart": dict(S=300, n=9, Hq=8, Hkv=2, P=8001, m=60, batched=False, plan=1, joined="memory"),
    "packed, ungrouped heads, apart": dict(S=300, n=3, Hq=4, Hkv=4, P=5000, m=100, batched=False, plan=1, joined="memory"),
    "batched, in the walk": dict(S=64, n=7, Hq=8, Hkv=2, P=8001, m=90, batched=True, plan=2, joined="memory"),
    "batched, in the walk, on the chip": dict(S=64, n=7, Hq=8, Hkv=2, P=2001, m=90, batched=True, plan=2, joined="chip"),
    "batched, half a tile each": dict(S=40, n=21, Hq=6, Hkv=2, P=9100, m=50, batched=True, plan=2, joined="chip"),
    "batched, apart": dict(S=70, n=5, Hq=16, Hkv=4, P=8001, m=64, batched=True, plan=1, joined="memory"),
}


class Call:
    """Inputs of a shape; lq, lk: lengths of the sequences (full: all of n and m)."""

    def __init__(self, name, full=False, mul=1.0):
        import bit_kv_cache_spc_gb300 as spc
        c = SHAPES[name]
        S, n, m, Hq, Hkv, P = (c[x] for x in ("S", "n", "m", "Hq", "Hkv", "P"))
        self.c, self.spc = c, spc
        # some without queries, some without keys, some with fewer keys than queries
        self.lq = [n if full or s % 3 == 0 else (s * 37) % (n + 1) for s in range(S)]
        self.lk = [m if full or s % 4 == 0 else (s * 53) % (m + 1) for s in range(S)]
        self.at = dict(q_len=i32(self.lq), k_len=i32(self.lk))
        if c["batched"]:  # queries of a padded batch, own keys in the head-major rows of caches
            self.q = rnd(1, S, n, Hq, D, mul=mul)
            self.k, self.v = (rnd(i, S, Hkv, m + 5, D, mul=x).transpose(1, 2) for i, x in ((2, mul), (3, 1.0)))
            self.rows = [self.q[s, :x] for s, x in enumerate(self.lq)]
        else:  # packed, with a gap within; own keys anywhere on their axis, shared here and there
            self.qb = [sum(self.lq[:s]) + 3 * (s > S // 2) for s in range(S)]
            self.kb = [(s * 131) % 300 for s in range(S)]
            self.q = rnd(1, S * n + 5, Hq, D, mul=mul)  # the same plan for all lengths
            self.k, self.v = (rnd(i, 300 + m, Hkv, D, mul=x) for i, x in ((2, mul), (3, 1.0)))
            self.at.update(q_begin=i32(self.qb), k_begin=i32(self.kb), q_max=n)
        self.at["k_max"] = m
        self.pk, self.pv = (rnd(i, Hkv, P + 3, D, mul=x)[:, :P].transpose(0, 1) for i, x in ((4, mul), (5, 1.0)))
        self.o, self.lse = torch.empty_like(self.q), torch.empty(self.q.shape[:-1], device="cuda")
        shape = (self.q, self.pk, self.pv, self.k, self.v, self.o)
        ask = dict(S=S, q_max=n, k_max=m)
        assert spc.spc_prefix_attn_together(*shape, **ask, placed=not c["batched"]) == c["plan"]
        assert (spc.spc_prefix_attn_workspace_bytes(*shape, **ask) > 256) == (c["joined"] == "memory")

    def run(self, **kw):
        self.o.fill_(7)
        self.lse.fill_(7)
        t = dict(pk=self.pk, pv=self.pv, k=self.k, v=self.v)
        t.update({x: kw.pop(x) for x in list(kw) if x in t})
        self.spc.spc_prefix_attn(self.q, t["pk"], t["pv"], t["k"], t["v"], self.o, self.lse, **self.at, **kw)
        return self.o, self.lse

    def of(self, x, s):
        """Sequence s's rows of a tensor that lies as the queries do."""
        return x[s, :self.lq[s]] if self.c["batched"] else x[self.qb[s]:self.qb[s] + self.lq[s]]

    def own(self, x, s):
        """And of one that lies as the keys do."""
        return x[s, :self.lk[s]] if self.c["batched"] else x[self.kb[s]:self.kb[s] + self.lk[s]]

    def check(self, P, some=1):
        used = torch.zeros(self.lse.shape[:-1], dtype=torch.bool, device="cuda")
        for s, (n, m) in enumerate(zip(self.lq, self.lk)):
            self.of(used, s)[:] = True
            if n and s % some == 0:
                k, v = torch.cat([self.pk[:P], self.own(self.k, s)]), torch.cat([self.pv[:P], self.own(self.v, s)])
                check(self.of(self.o, s), self.of(self.lse, s), self.of(self.q, s), k, v, prefix_sight(n, m, P))
        assert bool((self.o[~used] == 7).all()) and bool((self.lse[~used] == 7).all())
        assert not bool((self.lse[used] == 7).any())


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("name", SHAPES)
def test_lengths_that_differ(name, full):
    """Every row, and what belongs to no sequence left as it was; the same bits again."""
    c = Call(name, full)
    o, lse = (x.clone() for x in c.run())
    c.check(c.c["P"], some=1 if c.c["S"] <= 70 else 3)
    for _ in range(3):
        again = c.run()
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    assert c.spc.spc_prompt_attn_status() == 0


@pytest.mark.parametrize("length", [0, 1, 64, 100, 1407, -1, 1 << 20])
@pytest.mark.parametrize("name", SHAPES)
def test_a_length_of_the_prefix_on_the_device(name, length):
    """Shorter than the tensor, of no tokens, inside a block and a split, negative and beyond the tensor; what lies behind
    it holds NaN."""
    c = Call(name)
    P = max(0, min(length, c.c["P"]))
    c.pk[P:], c.pv[P:] = math.nan, math.nan
    c.run(p_len=i32([length]))
    c.check(P, some=2 if c.c["S"] <= 70 else 5)


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf, torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("name", SHAPES)
def test_other_sequences_keys_do_not_matter(name, what):
    """Own keys and values of every third sequence are poisoned: the others, in the same tiles, keep their bits."""
    c = Call(name)
    if not c.c["batched"]:  # keys of their own
        S, m = c.c["S"], c.c["m"]
        c.kb = [s * m for s in range(S)]
        c.k, c.v = (rnd(i, S * m, c.c["Hkv"], D) for i in (2, 3))
        c.at["k_begin"] = i32(c.kb)
    want = [x.clone() for x in c.run()]
    k, v = c.k.clone(), c.v.clone()
    for s in range(0, c.c["S"], 3):
        for x in (k, v):
            c.own(x, s)[:] = what
    got = c.run(k=k, v=v)
    for s in range(c.c["S"]):
        if s % 3:
            assert torch.equal(c.of(want[0], s), c.of(got[0], s)) and torch.equal(c.of(want[1], s), c.of(got[1], s)), s


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("name", SHAPES)
def test_rows_before_a_poisoned_key_do_not_see_it(name, what):
    """The last own key and value of every sequence: only its last query sees them, where it has as many keys as queries."""
    c = Call(name, full=True)
    S, n, m = c.c["S"], c.c["n"], c.c["m"]
    if not c.c["batched"]:
        c.kb = [s * m for s in range(S)]
        c.k, c.v = (rnd(i, S * m, c.c["Hkv"], D) for i in (2, 3))
        c.at["k_begin"] = i32(c.kb)
    want = [x.clone() for x in c.run()]
    k, v = c.k.clone(), c.v.clone()
    for s in range(S):
        for x in (k, v):
            c.own(x, s)[-1] = what
    got = c.run(k=k, v=v)
    for s in range(S):
        for x, y in zip(want, got):
            assert torch.equal(c.of(x, s)[:-1], c.of(y, s)[:-1]), s
        if not math.isinf(what):
            assert bool(torch.isnan(c.of(got[0], s)[-1]).all()), s


@pytest.mark.parametrize("name", SHAPES)
def test_visible_infinities_and_nan(name):
    """Values of the prefix, in its first block and its last, and of two sequences' own keys reach the rows that see them with
    their sign, and no others; all other channels keep their bits."""
    c = Call(name, full=True, mul=0.1)
    S, n, m, P = (c.c[x] for x in ("S", "n", "m", "P"))
    if not c.c["batched"]:
        c.kb = [s * m for s in range(S)]
        c.k, c.v = rnd(2, S * m, c.c["Hkv"], D, mul=0.1), rnd(3, S * m, c.c["Hkv"], D)
        c.at["k_begin"] = i32(c.kb)
    want = c.run()[0].clone()
    pv, v = c.pv.clone(), c.v.clone()
    pv[10, :, 3], pv[P - 3, :, 7], pv[P - 1, :, 9] = math.inf, -math.inf, math.nan
    c.own(v, 5)[m - 2, :, 11] = math.inf  # seen by the last two queries
    c.own(v, 5)[0, :, 13] = -math.inf     # by all from n - m on
    c.own(v, S - 1)[m - 1, :, 15] = math.nan  # by the last one
    got = c.run(pv=pv, v=v)[0]
    for s in range(S):
        o, w = c.of(got, s), c.of(want, s).clone()
        w[..., 3], w[..., 7], w[..., 9] = math.inf, -math.inf, math.nan
        if s == 5:
            w[-2:, :, 11] = math.inf
            w[max(0, n - m):, :, 13] = -math.inf
        if s == S - 1:
            w[-1:, :, 15] = math.nan
        assert torch.equal(torch.isnan(o), torch.isnan(w)) and torch.equal(o[~torch.isnan(o)], w[~torch.isnan(w)]), s


@pytest.mark.parametrize("name", SHAPES)
def test_captured_and_replayed_with_other_lengths(name):
    """Two graphs on one workspace, one behind the other, and then on two streams with a workspace each."""
    c = Call(name)
    P = i32([c.c["P"]])
    need = max(256, c.spc.spc_prefix_attn_workspace_bytes(c.q, c.pk, c.pv, c.k, c.v, c.o, S=c.c["S"], q_max=c.c["n"], k_max=c.c["m"]))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    want = [x.clone() for x in c.run(p_len=P, ws=ws)]
    torch.cuda.synchronize()
    first, second, o2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph(), torch.empty_like(c.o)
    call = lambda o, w, **kw: c.spc.spc_prefix_attn(c.q, c.pk, c.pv, c.k, c.v, o, c.lse, p_len=P, ws=w, **c.at, **kw)  # noqa: E731
    with torch.cuda.graph(first):
        call(c.o, ws)
    with torch.cuda.graph(second):
        call(o2, ws)
    c.o.fill_(7)
    o2.fill_(7)
    first.replay()
    second.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.o, want[0]) and torch.equal(o2, want[0]) and torch.equal(c.lse, want[1])
    P.fill_(777)
    c.lq = [n - 1 if n else 0 for n in c.lq]
    c.at["q_len"].copy_(i32(c.lq))
    c.o.fill_(7)
    c.lse.fill_(7)
    first.replay()
    torch.cuda.synchronize()
    c.check(777, some=4)
    P.fill_(c.c["P"])
    want = [x.clone() for x in c.run(p_len=P, ws=ws)]
    side, wss = [torch.cuda.Stream() for _ in range(2)], [torch.zeros_like(ws) for _ in range(2)]
    outs = [torch.full_like(c.o, 7.0) for _ in side]
    torch.cuda.synchronize()
    for _ in range(3):
        for st, o, w in zip(side, outs, wss):
            c.spc.spc_prefix_attn(c.q, c.pk, c.pv, c.k, c.v, o, p_len=P, ws=w, stream=st, **c.at)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) for o in outs)
    assert c.spc.spc_prompt_attn_status(ws) == 0 and c.spc.spc_prompt_attn_status() == 0
