"""spc_prefix_attn_together: which way a call behind a shared prefix goes, without a GPU."""
import ctypes as C

import pytest

from bit_kv_cache_spc_gb300 import _lib, spc_layout, spc_prefix, spc_prompt_dims
from test_gpu_prefix_together import SHAPES


def plan(S, n, m, Hq, Hkv, P, batched, axis=None, placed=0, **over):
    T = axis or (n if batched else S * n)
    ql = spc_layout(T * Hq * 128 if batched else 0, Hq * 128, 128)
    kl = spc_layout(m * Hkv * 128 if batched else 0, Hkv * 128, 128)
    d = spc_prompt_dims(S, Hq, Hkv, 128, T, m, n, m, 0.1, ql, kl, kl, ql)
    for x, y in over.items():
        setattr(d, x, y)
    pl = spc_layout(0, Hkv * 128, 128)
    p = spc_prefix(P, pl, pl)
    return (_lib.spc_prefix_attn_together(C.byref(d), C.byref(p), placed),
            _lib.spc_prefix_attn_workspace_bytes(C.byref(d), C.byref(p)))


@pytest.mark.parametrize("name", SHAPES)
def test_shapes_of_the_gpu_tests(name):
    c = dict(SHAPES[name])
    want, joined = c.pop("plan"), c.pop("joined")
    got, ws = plan(**c)
    assert got == want and (ws > 256) == (joined == "memory")
    assert plan(**c, placed=1)[0] == (0 if c["batched"] else want)


LIKE = dict(S=64, m=40, Hq=32, Hkv=8, P=8192)


def test_batched_queries_share_tiles_while_two_sequences_fit():
    assert plan(n=16, batched=True, **LIKE)[0] == 2 and plan(n=17, batched=True, **LIKE)[0] == 0
    assert plan(n=17, batched=False, **LIKE)[0] == 2


def test_packed_queries_share_tiles_on_an_axis_without_long_gaps():
    at = dict(LIKE, n=1, batched=False)
    assert plan(**at, axis=4 * 64)[0] == 1 and plan(**at, axis=4 * 64 + 1)[0] == 0


def test_single_tokens_always_share_them():
    for S in (2, 7, 500):
        for batched in (False, True):
            assert plan(**dict(LIKE, S=S, n=1, P=100, batched=batched))[0] == 1
    assert plan(**dict(LIKE, S=1, n=1, batched=False))[0] == 1


def test_others_walk_alone():
    at = dict(LIKE, n=7, batched=False)
    assert plan(**dict(at, S=1))[0] == 0 and plan(**dict(at, P=0))[0] == 0 and plan(**at, q_max=0)[0] == 0
    assert plan(**at, D=64) == (0, 0) and plan(**at, scale=0.0) == (0, 0)
    assert _lib.spc_prefix_attn_together(None, None, 0) == 0
