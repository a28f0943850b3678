"""More of the prompt path's host side: settings, and calls that are refused before anything reaches the GPU."""
import bit_kv_cache_spc_gb300 as spc


def test_the_wait_limit_is_read_and_set():
    assert spc.spc_prompt_attn_wait_limit() == 2_000_000_000
    try:
        assert spc.spc_prompt_attn_wait_limit(5) == 2_000_000_000
        assert spc.spc_prompt_attn_wait_limit(-1) == 5 and spc.spc_prompt_attn_wait_limit(0) == 5
    finally:
        assert spc.spc_prompt_attn_wait_limit(2_000_000_000) == 5
