"""A refused steps.prompt_layer leaves everything as it was, and may be made again with what it lacked."""
import pytest
import torch

pytestmark = pytest.mark.gpu
D, B, Hq, Hkv, R = 128, 2, 4, 2, 16


def rnd(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


class Layer:
    """A layer's cache after `before` tokens, and a prompt of n tokens for it."""

    def __init__(self, before, n):
        import bit_kv_cache_spc_gb300 as spc
        total = before + n
        self.spc, self.n, self.total = spc, n, total
        self.d = spc.Dims(B, Hq, Hkv, 0, R, 1, q_groups_cap=total // 32 + 1, resid_cap=R + 32)
        self.rec = torch.zeros(spc.spc_records_bytes(self.d), dtype=torch.uint8, device="cuda")
        self.res = torch.zeros(spc.spc_resid_bytes(self.d) // 2, dtype=torch.int16, device="cuda")
        self.host = torch.zeros((B, Hkv, total, 2, D), dtype=torch.int16, pin_memory=True)
        self.history = torch.zeros((2, B, Hkv, total, D), dtype=torch.bfloat16, device="cuda")
        self.turns = spc.spc_rope_frequencies(128)[0].cuda()
        if before:
            self.prompt(before, 1)
            self.run()
        self.prompt(n, 2)

    def prompt(self, n, seed):
        qkv = rnd(seed, B, n, Hq + 2 * Hkv, D)
        self.q, self.k, self.v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        self.pos = (self.d.N + torch.arange(n, device="cuda", dtype=torch.int32)).expand(B, n).contiguous()
        self.o = torch.zeros((B, n, Hq, D), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.zeros((B, n, Hq), device="cuda")

    def run(self, **other):
        from bit_kv_cache_spc_gb300.steps import prompt_layer
        a = dict(d=self.d, q=self.q, k=self.k, v=self.v, pos=self.pos, turns=self.turns, o=self.o, records=self.rec,
                 resid=self.res, host_kv=self.host, n_cap=self.total, history=self.history, lse=self.lse)
        prompt_layer(**{**a, **other})

    def state(self):
        torch.cuda.synchronize()
        return [x.clone() for x in (self.q, self.k, self.v, self.o, self.lse, self.rec, self.res, self.host, self.history)]


def shrunk(d, **caps):
    import bit_kv_cache_spc_gb300 as spc
    x = spc.spc_dims.from_buffer_copy(d)
    for name, value in caps.items():
        setattr(x, name, value)
    return x


BAD = {
    "records for too few groups": lambda s: dict(d=shrunk(s.d, q_groups_cap=s.total // 32 - 2)),
    "a window too small": lambda s: dict(d=shrunk(s.d, resid_cap=R - 1)),
    "host rows too few": lambda s: dict(n_cap=s.total - 1),
    "a host cache that is not pinned": lambda s: dict(host_kv=torch.zeros_like(s.host).clone()),
    "a cache without records": lambda s: dict(records=None),
    "a records tensor too small": lambda s: dict(records=s.rec[:-1]),
    "an output on the queries": lambda s: dict(o=s.q),
    "an lse of another shape": lambda s: dict(lse=s.lse[:, :-1].contiguous()),
    "positions of another shape": lambda s: dict(pos=s.pos[:, :-1].contiguous()),
    "a scale of zero": lambda s: dict(d=shrunk(s.d, scale=0.0)),
    "a misplaced window": lambda s: dict(resid=s.res.data_ptr() + 2),
}


@pytest.mark.parametrize("before", [0, 200])
@pytest.mark.parametrize("what", BAD)
def test_a_refused_prompt_changes_nothing(what, before):
    s, twin = Layer(before, 150), Layer(before, 150)
    was, N = s.state(), s.d.N
    bad = BAD[what](s)
    with pytest.raises((ValueError, s.spc.SpcError)):
        s.run(**bad)
    assert s.d.N == N and bad.get("d", s.d).N == N
    assert all(torch.equal(x, y) for x, y in zip(was, s.state()))
    s.run()  # made again, it is the prompt that was never refused
    twin.run()
    assert s.d.N == twin.d.N == N + 150
    assert all(torch.equal(x, y) for x, y in zip(s.state(), twin.state()))


def test_a_workspace_too_small_is_refused_before_the_rotation():
    """One token over a long history, whose keys are split."""
    s = Layer(6000, 1)
    was = s.state()
    with pytest.raises(s.spc.SpcError) as e:
        s.run(ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 5 and s.d.N == 6000
    assert all(torch.equal(x, y) for x, y in zip(was, s.state()))
    s.run()
    assert s.d.N == 6001


@pytest.mark.parametrize("before", [0, 200])
def test_a_prompt_of_no_tokens(before):
    s = Layer(before, 0)
    was = s.state()
    s.run()
    assert s.d.N == before
    assert all(torch.equal(x, y) for x, y in zip(was[:-1], s.state()[:-1]))
