"""spc_prompt_attn_status: one word of a workspace, three of the device, from several threads and beside a capture."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
D = 128
TIMEOUT = 6


def overrun(kind, ws=None):
    """A call whose waits run out (limit of a nanosecond), over half a million keys."""
    import bit_kv_cache_spc_gb300 as spc
    sms, keys = torch.cuda.get_device_properties(0).multi_processor_count, 1 << 19
    z = dict(dtype=torch.bfloat16, device="cuda")
    q, k = torch.zeros((2 * sms, 128, D), **z), torch.zeros((keys, 1, D), **z)
    v, o, own = torch.ones_like(k), torch.zeros_like(q), torch.zeros((2 * sms, 1, D), **z)
    before = spc.spc_prompt_attn_wait_limit(1)
    try:
        if kind == "plain":
            spc.spc_prompt_attn(q, k, v, o, ws=ws)
        elif kind == "window":
            spc.spc_window_attn(q, k, v, o, keys - 1, ws=ws)
        else:
            spc.spc_prefix_attn(q, k, v, own, own, o, ws=ws)
    finally:
        spc.spc_prompt_attn_wait_limit(before)


@pytest.mark.parametrize("kinds", [["plain"], ["window"], ["prefix"], ["prefix", "plain"], ["plain", "window", "prefix"]])
def test_each_kind_of_call_reports_to_the_device(kinds):
    import bit_kv_cache_spc_gb300 as spc
    spc.spc_prompt_attn_status()
    for kind in kinds:
        overrun(kind)
    assert spc.spc_prompt_attn_status() == TIMEOUT and spc.spc_prompt_attn_status() == 0


def test_a_workspace_has_its_own_word():
    import bit_kv_cache_spc_gb300 as spc
    ws = [torch.zeros(1 << 24, dtype=torch.uint8, device="cuda") for _ in range(2)]
    overrun("plain", ws[0])
    assert spc.spc_prompt_attn_status(ws[1]) == 0
    assert spc.spc_prompt_attn_status(ws[0]) == TIMEOUT and spc.spc_prompt_attn_status(ws[0]) == 0
    assert spc.spc_prompt_attn_status() == TIMEOUT and spc.spc_prompt_attn_status() == 0


def test_many_threads():
    """More at once than words are kept for; each finds what was written to its own workspace."""
    import bit_kv_cache_spc_gb300 as spc
    spc.spc_prompt_attn_status()
    ws = [torch.zeros(256, dtype=torch.uint8, device="cuda") for _ in range(24)]
    torch.cuda.synchronize()
    wrong, go = [], threading.Barrier(len(ws))

    def ask(i):
        st = torch.cuda.Stream()
        go.wait()
        for n in range(20):
            with torch.cuda.stream(st):
                if (n + i) % 3 == 0:
                    ws[i][:4].fill_(1)
                got = (spc.spc_prompt_attn_status(ws[i], stream=st), spc.spc_prompt_attn_status(ws[i], stream=st))
            if got != (TIMEOUT if (n + i) % 3 == 0 else 0, 0):
                wrong.append((i, n, got))

    threads = [threading.Thread(target=ask, args=(i,)) for i in range(len(ws))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and spc.spc_prompt_attn_status() == 0


def test_beside_a_capture():
    """A first call of another thread takes its words while a stream is being captured: the capture goes on.  (torch deals
    32 streams out by turns: 21 in a row are different ones.)"""
    import bit_kv_cache_spc_gb300 as spc
    captured, *streams = [torch.cuda.Stream() for _ in range(21)]
    assert len({s.cuda_stream for s in (captured, *streams)}) == 21
    ws, x = [torch.zeros(256, dtype=torch.uint8, device="cuda") for _ in range(20)], torch.zeros(64, device="cuda")
    torch.cuda.synchronize()
    got, go = [], threading.Barrier(len(ws))

    def ask(w, st):
        go.wait()
        got.append(spc.spc_prompt_attn_status(w, stream=st))

    threads = [threading.Thread(target=ask, args=a) for a in zip(ws, streams)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=captured, capture_error_mode="thread_local"):
        x.add_(1)
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        x.add_(1)
    g.replay()
    torch.cuda.synchronize()
    assert got == [0] * len(ws) and bool((x == 2).all())
