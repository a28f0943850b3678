"""Calls that start as the kernel before them ends, behind something else: copies, memsets and another stream's work in a graph,
and the same on streams."""
import pytest
import torch

from sight_ref import i32, rnd

pytestmark = pytest.mark.gpu
D = 128


def norm():
    import bit_kv_cache_spc_gb300 as spc
    q, w, turns = rnd(1, 2, 40, 8, D), 1 + rnd(2, D).float().abs(), spc.spc_rope_frequencies(128)[0].cuda()
    pos, o = torch.arange(80, dtype=torch.int32, device="cuda").view(2, 40), torch.zeros_like(q)
    return q, o, lambda: spc.spc_norm_rope(q, None, pos, turns, w, q_out=o)


def window(lq, lk, W):
    import bit_kv_cache_spc_gb300 as spc
    q, k, v = rnd(1, 2, lq, 8, D), rnd(2, 2, lk, 2, D), rnd(3, 2, lk, 2, D)
    o = torch.zeros_like(q)
    ws = torch.zeros(spc.spc_window_attn_workspace_bytes(q, k, v, o, W, 3), dtype=torch.uint8, device="cuda")
    return q, o, lambda: spc.spc_window_attn(q, k, v, o, W, 3, ws=ws)


def prefix(S, n, P):
    import bit_kv_cache_spc_gb300 as spc
    q, k, v, pk, pv = rnd(1, S, n, 16, D), rnd(2, S, 64, 4, D), rnd(3, S, 64, 4, D), rnd(4, P, 4, D), rnd(5, P, 4, D)
    o = torch.zeros_like(q)
    ws = torch.zeros(spc.spc_prefix_attn_workspace_bytes(q, pk, pv, k, v, o), dtype=torch.uint8, device="cuda")
    return q, o, lambda: spc.spc_prefix_attn(q, pk, pv, k, v, o, ws=ws)


CALLS = {"norm": norm, "window, single tokens": lambda: window(1, 900, 300), "window": lambda: window(50, 900, 300),
         "prefix, single tokens": lambda: prefix(9, 1, 3000), "prefix, in one walk": lambda: prefix(64, 7, 4001),
         "prefix, in two launches": lambda: prefix(70, 5, 8001), "prefix, alone": lambda: prefix(3, 90, 1000)}


def slow(x, n):
    """Work of some tens of microseconds on the current stream that leaves x as it is."""
    for _ in range(n):
        x = x.flip(0)
    return x if n % 2 == 0 else x.flip(0)


@pytest.mark.parametrize("before", ["copy", "memset", "kernel", "other stream", "both"])
@pytest.mark.parametrize("name", CALLS)
def test_behind_other_nodes(name, before):
    """The queries are written right before the call, by each kind of node, and its output is read right behind it; captured
    and replayed with other queries, and made on streams."""
    q, o, call = CALLS[name]()
    inputs = [q.clone(), rnd(77, *q.shape), torch.zeros_like(q)]
    want = []
    for x in inputs:
        q.copy_(x)
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        want.append(o.clone())
    src, got, pad = inputs[0].clone(), torch.zeros_like(o), torch.zeros(1 << 22, device="cuda")
    side = torch.cuda.Stream()

    def steps():
        main = torch.cuda.current_stream()
        if before == "copy":
            slow(pad, 3)
            q.copy_(src)
        elif before == "memset":
            q.view(torch.int16).zero_()  # all of them zeros
        elif before == "kernel":
            slow(pad, 3)
            torch.mul(src, 1.0, out=q)
        else:
            side.wait_stream(main)
            with torch.cuda.stream(side):
                slow(pad, 6)
                torch.mul(src, 1.0, out=q)
            if before == "both":
                slow(pad, 1)
            main.wait_stream(side)
        call()
        torch.mul(o, 1.0, out=got)

    same = lambda i: torch.equal(got, want[2 if before == "memset" else i])  # noqa: E731
    steps()
    torch.cuda.synchronize()
    assert same(0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        steps()
    for i in (1, 0, 1):
        src.copy_(inputs[i])
        q.fill_(3)
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert same(i), i
    for i in (0, 1, 0, 1):  # without waiting between them
        src.copy_(inputs[i])
        steps()
        assert same(i), i
