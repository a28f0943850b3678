"""Tables of axes given as arrays turn the pairs as the same lists do (spc_norm_rope, steps.prompt_layer)."""
import array

import numpy as np
import pytest
import torch

from test_gpu_norm_rope import check, rnd, weight
from test_gpu_prompt_layer_kinds import Model

pytestmark = pytest.mark.gpu
KINDS = [np.array, lambda x: np.array(x, dtype=np.int32), lambda x: array.array("i", x)]


@pytest.mark.parametrize("kind", KINDS)
def test_spc_norm_rope(kind):
    import bit_kv_cache_spc_gb300 as spc
    turns = spc.spc_rope_frequencies(128)[0]
    axis = spc.spc_rope_axes([24, 20, 20], 128, "turns")
    q, w = rnd(1, 2, 9, 4, 128), weight(2)
    pos = torch.randint(0, 1 << 16, (3, 2, 9), device="cuda", dtype=torch.int32)
    out = torch.empty_like(q)
    spc.spc_norm_rope(q, None, pos, turns.cuda(), w, axis=kind(axis), q_out=out)
    check(out, q, w, 1e-6, pos, turns, axis, 128, False)


@pytest.mark.parametrize("kind", KINDS)
def test_prompt_layer(kind):
    from bit_kv_cache_spc_gb300.steps import prompt_layer
    m = Model(1, 4, 2, 16, 1, 32, 40, 3)
    q, k, v, pos, o, lse = m.prompt(40)
    q0, k0 = q.clone(), k.clone()
    prompt_layer(m.d, q, k, v, pos, m.turns.cuda(), o, m.rec, m.res, lse=lse, **dict(m.norm(), axis=kind(m.axis)))
    m.check_rows(q, q0, m.wq, pos)
    m.check_rows(k, k0, m.wk, pos)
