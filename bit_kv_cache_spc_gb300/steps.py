"""The SpeCache page's per-layer steps (Algorithms 1-3) as sequences of the
library's C-ABI calls.

Nothing here computes: every step runs in libspc's kernels or copy-engine
copies; this module only orders the calls on the caller's streams and keeps
the cache length in the dims struct.

    prefill_layer   Algorithm 1: Quant(K), Quant(V) into the low-bit cache,
                    then Offload(C) of the 16-bit K/V to the pinned host cache
                    on a copy stream (section 3, "Prefilling").
    prompt_layer    Algorithm 1 from the projections on: rotary positions, the
                    prompt's causal attention, its K/V into the low-bit cache
                    and the host cache; also for the follow-up prompts of a
                    conversation, which attend over the cache read back.
    predecode_layer Algorithm 2: append the first token's K/V, attention of
                    its single query over the cache, ArgTopK over that
                    attention, Pre-fetch of the selected 16-bit rows.
    decode_layer    Algorithm 3: the append (and offload) of the real token's
                    K/V, the two-query attention over C' with the fetched rows
                    substituted, ArgTopK over the speculative row, Pre-fetch.
"""
from __future__ import annotations

import torch

from . import (_all_or_none, spc_append_kv, spc_decode_attn2, spc_dequantize_kv, spc_extend_kv, spc_host_gather,
               spc_host_gather_prev, spc_merged_attn, spc_offload_kv, spc_prompt_attn, spc_quantize_kv, spc_rope,
               spc_topk_select, spc_topk_select_prev)


def prefill_layer(d, k, v, records, resid, host_kv, n_cap, stream=None, copy_stream=None):
    """Quantise the layer's K and V (bf16 [B][Hkv][N][D], device) into
    records/resid on `stream`, and offload them to host_kv on `copy_stream`
    (default: `stream`).  Returns the event after which k and v may be freed."""
    stream = torch.cuda.current_stream() if stream is None else stream
    copy_stream = stream if copy_stream is None else copy_stream
    spc_quantize_kv(d, k, v, records, resid, stream=stream.cuda_stream)
    ready = torch.cuda.Event()
    ready.record(stream)
    copy_stream.wait_event(ready)
    spc_offload_kv(d, k, v, host_kv, n_cap, stream=copy_stream.cuda_stream)
    done = torch.cuda.Event()
    done.record(copy_stream)
    return done


def prompt_layer(d, q, k, v, pos, turns, o, records, resid, host_kv=None, n_cap=0, history=None, lse=None, ws=None,
                 rot=128, interleaved=False, mscale=1.0, stream=None):
    """A prompt of n tokens per sequence through one layer's attention, and
    into its cache.  q: 16-bit [B][n][Hq][D], k, v: [B][n][Hkv][D], views of
    the projections (any strides); pos: int32 [B][n], the tokens' positions;
    turns (and rot, interleaved, mscale): the rotary rule (spc_rope).  q is
    rotated in place.  o: [B][n][Hq][D]; lse: fp32 [B][n][Hq] or None.

    An empty cache (d.N = 0): k is rotated in place and the prompt attends to
    itself.  A follow-up prompt (d.N > 0) attends to the cache as well, read
    back in 16 bits: history is a pair of buffers [B][Hkv][cap][D] (keys,
    values) of cap >= d.N + n rows, which then hold the history's rows and the
    new tokens' behind them; they may be shared by layers that run in turn.
    The new tokens join records and resid, and host_kv if given; d.N is
    advanced by n.  The calls are checked in whole before the first one: one
    that is refused leaves q, k, history and the cache as they were, and may be
    made again.  Without ws the attention takes its workspace from torch's
    allocator; spc_prompt_attn_status(), after the layers, says whether a
    bounded wait of the attention ran out."""
    n, N = k.shape[1], d.N
    if N > 0:
        if history is None or any(b.shape[2] < N + n for b in history):
            raise ValueError(f"prompt_layer: a follow-up prompt needs history buffers of {N + n} rows")
        kk, vv = (b[:, :, :N + n].transpose(1, 2) for b in history)
    stream = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.stream(stream), _all_or_none() as calls:
        if N == 0:
            kk, vv = kn, vn = k, v
            spc_rope(q, k, pos, turns, rot, interleaved, mscale, _later=calls)
        else:
            kn, vn = kk[:, N:], vv[:, N:]
            spc_dequantize_kv(d, records, resid, 0, kk[:, :N], vv[:, :N], _later=calls)
            spc_rope(q, k, pos, turns, rot, interleaved, mscale, v=v, k_out=kn, v_out=vn, _later=calls)
        spc_prompt_attn(q, kk, vv, o, lse, scale=d.scale, ws=ws, _later=calls)
        spc_extend_kv(d, kn, vn, records, resid, host_kv, n_cap, _later=calls)
    d.N += n


def predecode_layer(d, records, resid, host_kv, n_cap, q1, k1, v1, k, idx, bitmap, staging, o, lse, logits, ws,
                    ws_bytes, q2, stream=None, fetch_stream=None):
    """Algorithm 2 for one layer.  q1: bf16 [B][Hq][D]; k1, v1: bf16
    [B][Hkv][D], the first generated token's rows.  The token's K/V joins the
    cache (d.N is advanced) and is offloaded to host_kv; the single query's
    attention is the two-query attention with both rows equal to q1 (q2 is a
    [B][2][Hq][D] scratch tensor), so its second row is the real token's and
    feeds ArgTopK.  The Pre-fetch runs on `fetch_stream` (default: `stream`)
    after the selection; the returned event marks its end."""
    stream = torch.cuda.current_stream() if stream is None else stream
    fetch_stream = stream if fetch_stream is None else fetch_stream
    s = stream.cuda_stream
    spc_append_kv(d, k1, v1, records, resid, host_kv, n_cap, stream=s)
    d.N += 1
    with torch.cuda.stream(stream):
        q2.copy_(q1.unsqueeze(1).expand(-1, 2, -1, -1))
    spc_decode_attn2(d, records, resid, q2, o, lse, logits, ws, ws_bytes, stream=s)
    spc_topk_select(d, logits, lse, k, idx, bitmap, stream=s)
    selected = torch.cuda.Event()
    selected.record(stream)
    fetch_stream.wait_event(selected)
    spc_host_gather(d, host_kv, n_cap, idx, k, staging, stream=fetch_stream.cuda_stream)
    fetched = torch.cuda.Event()
    fetched.record(fetch_stream)
    return fetched


def decode_layer(d, records, resid, host_kv, n_cap, q, k_t, v_t, k, idx, bitmap, staging, next_idx, next_bitmap,
                 next_staging, o, lse, logits, ws, ws_bytes, stream=None, fetch_stream=None, kv_self=None,
                 src=None):
    """Algorithm 3 for one layer.  The real token's K/V (k_t, v_t: bf16
    [B][Hkv][D]) first joins the cache and is offloaded (d.N is advanced), so
    both queries see it; q: bf16 [B][2][Hq][D] (the real token, then the
    speculative token).  idx/bitmap/staging hold the rows fetched for this
    step (selected at the previous step); the merged attention substitutes
    them, the speculative row's probabilities select next_idx/next_bitmap,
    and their Pre-fetch into next_staging runs on `fetch_stream`.  The
    speculative token's own K/V (kv_self: bf16 [B][Hkv][2][D], optional) is
    seen by the speculative query only and is not part of the cache.  With
    src (int32 [B][Hkv][k], scratch), the rows of the new selection that this
    step's selection already staged are copied from `staging` and only the
    others are read from the host (the used rows outside the new top-k are
    the ones evicted); next_staging is the same either way.  Returns the
    event that ends the Pre-fetch."""
    stream = torch.cuda.current_stream() if stream is None else stream
    fetch_stream = stream if fetch_stream is None else fetch_stream
    s = stream.cuda_stream
    spc_append_kv(d, k_t, v_t, records, resid, host_kv, n_cap, stream=s)
    d.N += 1
    spc_merged_attn(d, records, resid, q, idx, bitmap, staging, k, o, lse, logits, ws, ws_bytes, stream=s,
                    kv_self=kv_self)
    if src is None:
        spc_topk_select(d, logits, lse, k, next_idx, next_bitmap, stream=s)
    else:
        spc_topk_select_prev(d, logits, lse, k, next_idx, next_bitmap, idx, k, src, stream=s)
    selected = torch.cuda.Event()
    selected.record(stream)
    fetch_stream.wait_event(selected)
    if src is None:
        spc_host_gather(d, host_kv, n_cap, next_idx, k, next_staging, stream=fetch_stream.cuda_stream)
    else:
        spc_host_gather_prev(d, host_kv, n_cap, next_idx, k, next_staging, src, staging, k,
                             stream=fetch_stream.cuda_stream)
    fetched = torch.cuda.Event()
    fetched.record(fetch_stream)
    return fetched
