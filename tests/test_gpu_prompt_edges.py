"""Calls at the edges of what the prompt path takes."""
import pytest
import torch

pytestmark = pytest.mark.gpu
D = 128


def rnd(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def test_a_workspace_that_is_none_is_refused():
    """An expanded tensor's elements are not memory; an address alone says nothing of its size."""
    import bit_kv_cache_spc_gb300 as spc
    q, k, v = rnd(1, 1, 8, D), rnd(2, 4000, 2, D), rnd(3, 4000, 2, D)
    o = torch.full_like(q, 7.0)
    need = spc.spc_prompt_attn_workspace_bytes(q, k, v, o)
    assert need > 256
    room = torch.zeros(2 * need, dtype=torch.uint8, device="cuda")
    for ws in (room[:1].expand(need), room[::2], room.data_ptr(), room.cpu()):
        with pytest.raises(ValueError):
            spc.spc_prompt_attn(q, k, v, o, ws=ws)
    assert bool((o == 7).all())
    spc.spc_prompt_attn(q, k, v, o, ws=room.data_ptr(), ws_bytes=need)
    got = o.clone()
    spc.spc_prompt_attn(q, k, v, o)
    assert torch.equal(got, o)


def test_rows_of_no_elements_are_refused():
    import bit_kv_cache_spc_gb300 as spc
    x = torch.zeros((4, 2, 0), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        spc.spc_prompt_attn(x, x, x, torch.zeros_like(x))
