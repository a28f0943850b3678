/*
 * spc.h -- C ABI of libspc, the GB300 (sm_103a) decode-time hot path of
 * SpeCache ("SpeCache: Speculative Key-Value Caching for Efficient Generation
 * of LLMs", arXiv 2503.16163).
 *
 * The library implements the per-layer primitives the page's Algorithms 1-3
 * name: Quant (section 3), Attn over [T_t, T'_{t+1}] with C' U C_kappa
 * (section 3 "Decoding", Algorithm 3), ArgTopK over the speculative token's
 * attention row (Algorithm 3; Algorithm 2 for the pre-decoding step) and
 * Pre-fetch of the selected 16-bit rows from CPU memory (Algorithm 3).
 *
 * Conventions for every call:
 *   - Pointers are device pointers unless stated otherwise; bf16 values are
 *     passed as their 16-bit patterns (uint16_t).  All tensors are dense,
 *     row-major, and 16-byte aligned.
 *   - The caller owns and allocates every buffer.  The library never
 *     allocates, frees or synchronises; each call enqueues its kernels on the
 *     given stream (NULL = the legacy default stream) and returns.
 *   - Calls are stateless and may be made from several host threads.
 *   - Argument errors return SPC_ERR_INVALID / SPC_ERR_UNSUPPORTED before
 *     anything is launched; a failed launch returns SPC_ERR_CUDA (the CUDA
 *     error is left for cudaGetLastError / spc_last_cuda_error).
 */
#ifndef SPC_H
#define SPC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SPC_ABI_VERSION 2

/* A cudaStream_t. */
typedef struct CUstream_st* spc_stream;

typedef enum spc_status {
  SPC_OK = 0,
  SPC_ERR_INVALID = 1,     /* bad argument (null pointer, size, alignment) */
  SPC_ERR_UNSUPPORTED = 2, /* valid shape this build does not handle */
  SPC_ERR_CUDA = 3,        /* a CUDA runtime call or kernel launch failed */
  SPC_ERR_NOT_MAPPED = 4,  /* host pointer is not device-mapped pinned memory */
  SPC_ERR_WORKSPACE = 5,   /* workspace smaller than the size query returns */
  SPC_ERR_TIMEOUT = 6      /* a bounded wait inside a kernel ran out (spc_read_device_status) */
} spc_status;

/*
 * Shape of one layer's cache.  D must be 128 and group g 32 or 64 (the page's
 * group sizes, section 4 and the appendix's LongBench runs).  G = Hq / Hkv
 * query heads share a KV head; this build handles G in {1, 2, 4}.
 * The quantised prefix has N_q = floor(max(N - R, 0) / g) * g tokens and the
 * residual window the last r = N - N_q tokens (KIVI keeps the most recent
 * tokens in 16 bits; SpeCache page, section 4).  Capacities bound the buffers:
 * N_q / 32 <= q_groups_cap and r <= resid_cap.
 */
typedef struct spc_dims {
  int32_t B, Hq, Hkv, D;
  int32_t bits;         /* 1 or 2 */
  int32_t group;        /* g: 32 or 64 */
  int32_t N;            /* visible tokens of this layer */
  int32_t R;            /* residual window target */
  int32_t q_groups_cap; /* 32-token groups the record array can hold per (b,hkv) */
  int32_t resid_cap;    /* residual rows the residual buffer can hold per (b,hkv) */
  float scale;          /* softmax scale applied to q.k, e.g. 1/sqrt(128) */
} spc_dims;

int32_t spc_abi_version(void);
const char* spc_status_string(spc_status s);
/* The cudaError_t of the last SPC_ERR_CUDA on this host thread (0 if none). */
int32_t spc_last_cuda_error(void);

/* N_q of the shape (see spc_dims).  Returns -1 for an invalid shape. */
int32_t spc_num_quantized(const spc_dims* d);

/*
 * Low-bit copy C' of one layer ("records").  Bytes spc_records_bytes(d) in
 * all, row-major [B][Hkv][records per (b, hkv)][record bytes].
 *
 * g = 32: per (b, hkv) q_groups_cap records of 1024*(bits+1) bytes; record g
 * holds tokens 32g .. 32g+31 and is, in order:
 *   K codes  : `bits` planes of 128 u32 words (plane p holds bit p of each code)
 *   K minmax : 128 u32 words, min in bits 0..15 and max in bits 16..31 (bf16)
 *   V codes  : `bits` planes of 128 u32 words
 *   V minmax : 128 u32 words
 * With L = 4a + t (a in 0..7, t in 0..3), j in 0..3 and bit b in 0..31:
 *   K code word 4L+j, bit b : with v = (b + 21) mod 32, n = v mod 4,
 *                             q = v div 4, i = (4 - q mod 4) mod 4,
 *                             h = 1 if 1 <= q <= 4 else 0, e = 4j + i:
 *                             token 8n + a, channel 16*(e>>1) + 8*(e&1) + 2t + h
 *                             (rotated left by 4i, the word holds token 8n + a's
 *                             bits for channels 16*(e>>1) + 8*(e&1) + 2t + {0, 1}
 *                             at bits 11 + n and 27 + n)
 *   K minmax word 32t+m     : channel 16*(m>>2) + 2t + 8*((m>>1)&1) + (m&1)
 *   V code word 4L+j, bit b : token 16*(j>>1) + 8*(j&1) + 2t + (b>>4),
 *                             channel 16*((b&15)>>1) + 8*(b&1) + a
 *   V minmax word 32t+m     : token 16*(m>>4) + 8*((m>>3)&1) + 2t + ((m>>2)&1),
 *                             channel group m&3
 * This is 64 (1-bit) or 96 (2-bit) bytes per token and KV head, 1/8 or 3/16
 * of bf16.
 *
 * g = 64: per (b, hkv) (q_groups_cap + 1) / 2 records of 2048*bits + 1024
 * bytes; record u holds the 64-token group of tokens 64u .. 64u+63 as two
 * halves H = 0, 1 (tokens 64u + 32H ..), each group's metadata stored once:
 *   K codes of half 0, then of half 1 (`bits` planes of 128 words each, the
 *              code word rule above for the half's 32 tokens)
 *   K minmax : 128 words, word 32t+m as above, extremes over the 64 tokens
 *   V codes of half 0, then of half 1 (as above)
 *   V minmax : 128 words; word 64H + 2m + c holds token 32H + 16*((m>>2)&1) +
 *              8*((m>>1)&1) + 2*(m>>3) + (m&1) of the record, channels
 *              64c .. 64c+63
 * This is 48 (1-bit) or 80 (2-bit) bytes per token and KV head.
 *
 * Keys are grouped per channel over g tokens, values per token over g
 * consecutive channels (KIVI's axes).  min/max are the group's exact bf16
 * extremes (-0.0 stored as +0.0); the zero point and scale are derived from
 * them (SpeCache page, section 3): 1-bit z = (3min+max)/4, s = (max-min)/2;
 * 2-bit z = min, s = (max-min)/3.
 */
size_t spc_records_bytes(const spc_dims* d);

/* Residual window: bf16 [B][Hkv][resid_cap][2][D]; row j holds the key then
 * the value of token N_q + j.  The same [.., 2, D] row format is used for the
 * full 16-bit host cache and for the staging buffer of fetched rows. */
size_t spc_resid_bytes(const spc_dims* d);

/*
 * Quant (SpeCache page, section 3; Algorithm 1, K' = Quant(K), V' = Quant(V)).
 * k, v: bf16 [B][Hkv][N][D] (device).  Writes records 0 .. N_q/g-1 of every
 * (b,hkv) and residual rows 0 .. r-1.  Codes are
 *   clamp(rint((x - z) / s), 0, 2^bits - 1), code 0 when s == 0,
 * with z, s and (x - z) / s evaluated in IEEE binary32, round to nearest even,
 * without fused multiply-add.
 */
spc_status spc_quantize_kv(const spc_dims* d, const uint16_t* k, const uint16_t* v,
                           void* records, uint16_t* resid, spc_stream stream);

/* Bytes of device workspace spc_decode_attn2 / spc_merged_attn need for this
 * shape on the current device with at most k_max fetched rows per (b, hkv):
 * control words (three per (b, hkv) and a fault word, padded to 256 bytes)
 * followed by the split-K partials (one per CTA of the attention grid and
 * query row, merged by the call's second kernel unless the CTAs combine in a
 * cluster).  The caller zero-fills a workspace once after allocating it;
 * every call leaves the control words zero again.  Calls that share a
 * workspace must not overlap on the GPU (issue them on one stream, or order
 * them with events).
 * Returns 0 for an invalid shape. */
size_t spc_attn_workspace_bytes(const spc_dims* d, int32_t k_max);

/*
 * Attn([T_t, T'_{t+1}], C') -- the two-query decode attention over the
 * low-bit copy (SpeCache page, section 3 "Decoding"; with no fetched rows this is also
 * the pre-decoding attention of Algorithm 2).
 *   q     : bf16 [B][2][Hq][D]; row 0 is the output token T_t, row 1 the
 *           speculative token T'_{t+1}.  Query head h uses KV head h / G.
 *   kv_self : bf16 [B][Hkv][2][D] (per (b, hkv) the key row, then the value
 *           row) or NULL: the speculative token's own key and value, seen by
 *           the speculative query only (it follows T_t, so T_t does not see
 *           it), as one more visible row that is not a cache position (no
 *           spec_logits entry, never selected; its probability still counts
 *           in the speculative lse).  Algorithm 3 attends over [K, K_t] with
 *           the new tokens' rows; the speculative token's row cannot join the
 *           cache, so it is passed here and dropped after the call.
 *   o     : bf16 [B][2][Hq][D], softmax(scale * q.K^T) V over all N tokens
 *           (and the speculative row's own row for q row 1), keys/values
 *           dequantised from C' for n < N_q, residual rows after.
 *   lse   : fp32 [B][2][Hq] or NULL, natural log of the softmax normaliser.
 *   spec_logits : fp32 [B][Hkv][G][q_groups_cap*32] or NULL: the speculative
 *           token's scaled logits scale*q.k at the quantised positions, the
 *           input of spc_topk_select.
 *   ws    : zero-filled-once device workspace of at least
 *           spc_attn_workspace_bytes(d, 0) bytes (see that function).
 */
spc_status spc_decode_attn2(const spc_dims* d, const void* records, const uint16_t* resid,
                            const uint16_t* q, const uint16_t* kv_self, uint16_t* o, float* lse,
                            float* spec_logits, void* ws, size_t ws_bytes, spc_stream stream);

/*
 * Attn([T_t, T'_{t+1}], C' U C_kappa) (SpeCache page, section 3 "Decoding",
 * Algorithm 3): as spc_decode_attn2, but at the k positions idx[b][hkv][0..k-1]
 * (ascending, < N_q, -1 entries ignored) both the key and the value are the
 * fetched 16-bit rows staging[b][hkv][j] (bf16 [B][Hkv][k][2][D]) instead of
 * the low-bit rows.  bitmap (u32 [B][Hkv][q_groups_cap], bit n%32 of word
 * n/32) must mark exactly the listed positions.  spec_logits at a fetched
 * position holds the logit of the fetched row.  k = 0 is spc_decode_attn2.
 * ws holds at least spc_attn_workspace_bytes(d, k) bytes.
 */
spc_status spc_merged_attn(const spc_dims* d, const void* records, const uint16_t* resid,
                           const uint16_t* q, const uint16_t* kv_self, const int32_t* idx, const uint32_t* bitmap,
                           const uint16_t* staging, int32_t k, uint16_t* o, float* lse,
                           float* spec_logits, void* ws, size_t ws_bytes, spc_stream stream);

/*
 * Attn([T_t, T'_{t+1}], C' U C_kappa) of one layer together with the
 * Pre-fetch(C_kappa) of another layer (SpeCache page section 3, Algorithm 3:
 * the prefetch runs "in parallel with the following layers' computation").
 * Same as spc_merged_attn, and in the same launch the selected 16-bit rows
 * fetch_idx ([B][Hkv][fetch_k], same B and Hkv) of the pinned, mapped host
 * cache fetch_host_kv ([B][Hkv][fetch_n_cap][2][D], HOST pointer) are copied
 * to fetch_staging ([B][Hkv][fetch_k][2][D]), exactly as spc_host_gather
 * would.  The copy rides on the attention's own load pipeline, so the host
 * link works while the SMs compute; the attention's results are unchanged.
 * fetch_staging must not share a byte with the staging rows this call reads
 * (SPC_ERR_INVALID: the copy would race with the attention's reads).
 * fetch_k = 0 is spc_merged_attn.  SPC_ERR_NOT_MAPPED as spc_host_gather.
 */
spc_status spc_merged_attn_fetch(const spc_dims* d, const void* records, const uint16_t* resid,
                                 const uint16_t* q, const uint16_t* kv_self, const int32_t* idx,
                                 const uint32_t* bitmap,
                                 const uint16_t* staging, int32_t k, uint16_t* o, float* lse, float* spec_logits,
                                 void* ws, size_t ws_bytes, const uint16_t* fetch_host_kv, int64_t fetch_n_cap,
                                 const int32_t* fetch_idx, int32_t fetch_k, uint16_t* fetch_staging,
                                 spc_stream stream);

/*
 * spc_merged_attn_fetch that keeps the rows already staged (SpeCache page,
 * section 3, pre-fetching and offloading during decoding: the 16-bit rows
 * that are not in the new top-k are evicted, so the rows that are stay).
 * Row j of the new selection, fetch_idx[b][hkv][j], is copied from
 * fetch_prev_staging[b][hkv][fetch_src[b][hkv][j]] (device,
 * [B][Hkv][fetch_prev_k][2][D]) when fetch_src[b][hkv][j] >= 0, else from
 * the host cache; fetch_src is what spc_topk_select_prev writes for this
 * selection against the previous one, whose rows fetch_prev_staging holds.
 * fetch_staging is then exactly what spc_merged_attn_fetch writes, with only
 * the new rows read over the host link.  fetch_prev_staging must not share
 * a byte with fetch_staging (16-byte aligned; NULL only with fetch_prev_k = 0, when
 * every row comes from the host).  Everything else as spc_merged_attn_fetch.
 */
spc_status spc_merged_attn_fetch_prev(const spc_dims* d, const void* records, const uint16_t* resid,
                                      const uint16_t* q, const uint16_t* kv_self, const int32_t* idx,
                                      const uint32_t* bitmap, const uint16_t* staging, int32_t k, uint16_t* o,
                                      float* lse, float* spec_logits, void* ws, size_t ws_bytes,
                                      const uint16_t* fetch_host_kv, int64_t fetch_n_cap, const int32_t* fetch_idx,
                                      int32_t fetch_k, uint16_t* fetch_staging, const int32_t* fetch_src,
                                      const uint16_t* fetch_prev_staging, int32_t fetch_prev_k, spc_stream stream);

/*
 * Kernels that spc_decode_attn2 (k = 0), spc_merged_attn (k > 0) or
 * spc_merged_attn_fetch (fetch_k > 0) enqueue for this shape on the current
 * device: 1 when the CTAs of every (b, hkv) form one resident thread-block
 * cluster and combine their split-K partials through distributed shared
 * memory, else 2 (the attention grid stores its partials in the workspace and
 * a second, small kernel merges them).  A host-side query (no launch), for
 * callers that count launches or plan CUDA graphs.  -1 for an invalid shape
 * or a negative count.
 */
int32_t spc_attn_kernel_count(const spc_dims* d, int32_t k, int32_t fetch_k);

/*
 * One decoding step of a layer (SpeCache page, Algorithm 3) in one launch:
 * spc_merged_attn (optionally carrying another layer's Pre-fetch, as
 * spc_merged_attn_fetch) followed by ArgTopK(A_{1,:}), exactly as
 * spc_topk_select(d, spec_logits, lse, next_k, next_idx, next_bitmap) would
 * compute it.  The selection runs at the end of the attention: the CTA that
 * combines a (b, hkv) publishes its log-sum-exp, every CTA of the (b, hkv)
 * waits for it (bounded by a timer; on expiry it sets a fault word, reported
 * by spc_read_device_status) and keeps its chunk's candidates, and the last
 * CTA selects the final next_k.  So the speculative logits are re-read from
 * L2 by the CTAs that wrote them instead of by a second kernel.
 *   next_idx, next_bitmap: outputs as spc_topk_select's; they may be the idx
 *            and bitmap this call reads (every CTA of a (b, hkv) has read them
 *            before any is written).
 *   ws, ws_bytes: at least spc_step_workspace_bytes(d, max(k, next_k)),
 *            zero-filled once (the same contract as spc_attn_workspace_bytes).
 *   lse is required (non-NULL).
 *   spec_logits: as spc_merged_attn's, or NULL to keep the speculative
 *            logits on chip: every CTA then holds its chunk's logits in its
 *            SM's tensor memory (TMEM, 128 of the SM's 512 columns, lane =
 *            token, column = head) from the low-bit loop to its selection, so
 *            they are neither written to nor read back from device memory;
 *            only the fetched rows' logits (k x 4 floats per (b, hkv)) pass
 *            through the workspace.  The selection is identical.  NULL is
 *            accepted when spc_decode_step_on_chip returns 1 for the same
 *            arguments, else the call returns SPC_ERR_UNSUPPORTED.
 *   fetch_*: as spc_merged_attn_fetch; fetch_k = 0 for none.
 * Every CTA of the launch must be resident at once (the attention's grid is
 * one wave of the GPU): if other work holds the SMs for long enough, the
 * waits run out and the selection is wrong (SPC_ERR_TIMEOUT from
 * spc_read_device_status; zero-fill the workspace again before reuse).  When
 * the selection does not fit the attention's shared memory it is launched
 * separately, right after, on the same stream, with the same results.
 */
size_t spc_step_workspace_bytes(const spc_dims* d, int32_t k_max);
/* 1 when spc_decode_step with these arguments can keep the speculative logits
 * on chip (spec_logits == NULL): the selection rides on the attention launch
 * (k > 0) and each warp's 32-token groups need at most 32 x 4 TMEM columns.
 * 0 otherwise, -1 for an invalid shape or a negative count.  A host-side query. */
int32_t spc_decode_step_on_chip(const spc_dims* d, int32_t k, int32_t fetch_k, int32_t next_k);
/* Kernels one spc_decode_step with these arguments enqueues on the current
 * device: 1 when the selection rides on the attention launch, else the
 * attention's (spc_attn_kernel_count) plus the separate top-k.  -1 for an
 * invalid shape or a negative count. */
int32_t spc_decode_step_kernel_count(const spc_dims* d, int32_t k, int32_t fetch_k, int32_t next_k);
spc_status spc_decode_step(const spc_dims* d, const void* records, const uint16_t* resid, const uint16_t* q,
                           const uint16_t* kv_self, const int32_t* idx, const uint32_t* bitmap, const uint16_t* staging, int32_t k,
                           uint16_t* o, float* lse, float* spec_logits, int32_t next_k, int32_t* next_idx,
                           uint32_t* next_bitmap, void* ws, size_t ws_bytes, const uint16_t* fetch_host_kv,
                           int64_t fetch_n_cap, const int32_t* fetch_idx, int32_t fetch_k,
                           uint16_t* fetch_staging, spc_stream stream);

/*
 * spc_decode_step with the staged rows kept, as spc_merged_attn_fetch_prev
 * and spc_topk_select_prev do separately: the carried pre-fetch copies the
 * rows that fetch_src places in fetch_prev_staging ([B][Hkv][fetch_prev_k][2][D],
 * device) and reads only the others from the host, and the selection also
 * writes next_src ([B][Hkv][next_k]): each selected position's index in idx
 * (this call's own selection, k entries), else -1.  fetch_src is required when
 * fetch_k > 0; fetch_prev_staging must not share a byte with fetch_staging,
 * nor fetch_staging with staging, and next_idx none with idx here (next_src
 * is read against idx after next_idx is written): SPC_ERR_INVALID.
 * Everything else as spc_decode_step; outputs identical to it and to the
 * separate calls.
 */
spc_status spc_decode_step_prev(const spc_dims* d, const void* records, const uint16_t* resid, const uint16_t* q,
                                const uint16_t* kv_self, const int32_t* idx, const uint32_t* bitmap,
                                const uint16_t* staging, int32_t k, uint16_t* o, float* lse, float* spec_logits,
                                int32_t next_k, int32_t* next_idx, uint32_t* next_bitmap, int32_t* next_src,
                                void* ws, size_t ws_bytes, const uint16_t* fetch_host_kv, int64_t fetch_n_cap,
                                const int32_t* fetch_idx, int32_t fetch_k, uint16_t* fetch_staging,
                                const int32_t* fetch_src, const uint16_t* fetch_prev_staging, int32_t fetch_prev_k,
                                spc_stream stream);

/*
 * Reads and clears the fault word of an attention workspace (ws, laid out for
 * d): SPC_ERR_TIMEOUT if a bounded wait of spc_decode_step ran out since the
 * last read, else SPC_OK.  Synchronises `stream`.
 */
spc_status spc_read_device_status(void* ws, const spc_dims* d, spc_stream stream);

/*
 * spc_merged_attn without a caller-provided workspace.  The SpeCache paper has
 * no counterpart to this call; it exists for callers that cannot allocate
 * device memory (a plug-in running inside a host that owns the device
 * allocator, or a path where cudaMalloc's implicit synchronisation is not
 * allowed).  Same arguments and results as spc_merged_attn minus kv_self
 * (none) and ws/ws_bytes:
 * the workspace is a fixed 8 MiB buffer compiled into the library, which each
 * GPU that uses this call holds until the process exits.  Nothing is
 * allocated.  Argument errors return the statuses spc_merged_attn returns,
 * before anything is enqueued.  The buffer's device address is looked up
 * (cudaGetSymbolAddress) on the first call in each CUDA context and kept for
 * that context (a context made after a device reset gets a fresh lookup), so
 * make that first call before any stream capture.  Shapes whose workspace
 * (spc_attn_workspace_bytes(d, k)) exceeds 8 MiB return SPC_ERR_WORKSPACE.
 * All calls share the buffer: calls that overlap on the GPU race, so issue
 * them in order on one stream.
 */
spc_status spc_merged_attn_noalloc(const spc_dims* d, const void* records, const uint16_t* resid,
                                   const uint16_t* q, const int32_t* idx, const uint32_t* bitmap,
                                   const uint16_t* staging, int32_t k, uint16_t* o, float* lse,
                                   float* spec_logits, spc_stream stream);

/*
 * Offload(C) (SpeCache page, section 3 "Prefilling", Algorithm 1): after a
 * layer's attention the full-precision K and V (device, bf16 [B][Hkv][N][D]
 * each) are copied to the pinned host cache host_kv (HOST pointer, bf16
 * [B][Hkv][n_cap][2][D], rows interleaved K then V; pinned and mapped,
 * otherwise SPC_ERR_NOT_MAPPED; n_cap >= N), so that the device can release
 * them before the next layer.  Rows n < N are written; the copy engines do
 * the work (two strided copies per (b, hkv)), asynchronously on `stream`,
 * typically a copy stream overlapped with the next layer's compute.
 */
spc_status spc_offload_kv(const spc_dims* d, const uint16_t* k, const uint16_t* v, uint16_t* host_kv,
                          int64_t n_cap, spc_stream stream);

/*
 * Where the elements of a [batch][token][head][D] tensor lie: strides in
 * elements (bf16); the D elements of a head's row are contiguous.  Strides are
 * multiples of 8 (rows on 16-byte boundaries); t and h are positive, b is not
 * negative, and no two rows share a byte.  The calls below take such views, so
 * that projections are used where they are: a fused projection
 * [B][T][Hq + 2 Hkv][D] is three views of it, and a cache buffer
 * [B][Hkv][cap][D] is the view {Hkv*cap*D, D, cap*D}.  Their int32 and fp32
 * arrays lie on 4-byte boundaries (SPC_ERR_INVALID otherwise).
 */
typedef struct spc_layout {
  int64_t b, t, h;
} spc_layout;

/*
 * Rotary positions.  Pair i (0 <= i < rot/2) of a head's row at position p is
 * turned by the angle p * f_i and scaled by mscale:
 *   (x, y) -> mscale * (x cos - y sin, x sin + y cos),
 * elements rot..D-1 stay as they are.  Pairs are (i, i + rot/2) (the half
 * layout) or (2i, 2i + 1) (interleaved).  The frequencies are kept as 64-bit
 * fractions of a turn per position, turns[i] = 2^64 f_i / 2 pi: the angle is
 * the integer product p * turns[i] mod 2^64, exact at any position, so far
 * positions lose nothing.
 */
typedef enum spc_rope_kind {
  SPC_ROPE_PLAIN = 0,  /* f_i = theta^(-2i/rot) */
  SPC_ROPE_LINEAR = 1, /* f_i / factor (positions stretched) */
  SPC_ROPE_BANDS = 2,  /* by the pair's turns within context positions: at least high: f_i; at most low:
                          f_i / factor; between, the straight mix of the two in the number of turns */
  SPC_ROPE_RAMP = 3    /* by the pair's index ("YaRN", arXiv 2309.00071): f_i up to the pair that makes `high`
                          turns within context (rounded down), f_i / factor from the one that makes `low` on
                          (rounded up), a straight ramp between; mscale = 0.1 ln(factor) + 1 */
} spc_rope_kind;

typedef struct spc_rope_scaling {
  int32_t kind;     /* spc_rope_kind */
  double theta;     /* base, > 1 */
  double factor;    /* >= 1; not PLAIN */
  double low, high; /* BANDS, RAMP: numbers of turns, 0 < low < high (e.g. 1 and 4; 1 and 32) */
  double context;   /* BANDS, RAMP: positions of the unscaled context, > 0 */
} spc_rope_scaling;

/* Fills turns (HOST, rot/2 words; the caller uploads them once) and mscale
 * (HOST) for a rule.  A host-side computation in binary64. */
spc_status spc_rope_frequencies(const spc_rope_scaling* s, int32_t rot, uint64_t* turns, float* mscale);

typedef struct spc_rope_dims {
  int32_t B, T, Hq, Hkv, D; /* D = 128 */
  int32_t rot;              /* rotated elements of a head: a multiple of 16, 16 .. 128 */
  int32_t interleaved;      /* 0: pairs (i, i + rot/2); 1: pairs (2i, 2i + 1) */
  float mscale;             /* finite; 1 for most rules */
  spc_layout q, k, v, q_out, k_out, v_out;
} spc_rope_dims;

/*
 * Rotates T tokens' query and key rows, and copies their value rows, from the
 * projection to where they are used (the cache's rows, say), in one launch.
 *   pos    : int32 [B][T] (device), each token's position; any int32.
 *   turns  : uint64 [rot/2] (device).
 *   q, k   : bf16 views [B][T][Hq][D] and [B][T][Hkv][D]; v [B][T][Hkv][D] or
 *            NULL (no values).  Either of q and k may be NULL with Hq or
 *            Hkv 0 (v needs Hkv).
 *   *_out  : where the rows go; in place when pointer and layout equal the
 *            input's, else sharing no byte range with it.  No output row may
 *            share a byte with another tensor's rows (SPC_ERR_INVALID; views of
 *            different strides that reach into one another are only compared
 *            by their first rows).
 * Products and sums are binary32 (fused), rounded once to bf16.
 */
spc_status spc_rope(const spc_rope_dims* d, const int32_t* pos, const uint64_t* turns, const uint16_t* q,
                    const uint16_t* k, const uint16_t* v, uint16_t* q_out, uint16_t* k_out, uint16_t* v_out,
                    spc_stream stream);

/*
 * Which axis of the positions turns each pair, for positions of several axes
 * (time, height and width of a video's tokens, say).  sections (HOST, `axes`
 * numbers >= 0, in sum rot/2): how many pairs each axis turns.  Fills axis
 * (HOST, rot/2 bytes).
 */
typedef enum spc_axis_order {
  SPC_AXIS_SECTIONS = 0, /* the first sections[0] pairs axis 0, the next sections[1] axis 1, and so on */
  SPC_AXIS_TURNS = 1     /* pair i axis a = i % axes where i < axes * sections[a], else axis 0 (SPC_ERR_INVALID where an
                            axis then turns another number of pairs than its section says) */
} spc_axis_order;

spc_status spc_rope_axes(const int32_t* sections, int32_t axes, int32_t order, int32_t rot, uint8_t* axis);

typedef struct spc_norm_rope_dims {
  spc_rope_dims rope;
  int32_t axes;     /* of the positions: 1 .. 4 */
  float eps;        /* finite, at least 1e-30 (read where there is a weight) */
  uint8_t axis[64]; /* of each pair i < rot/2: below axes */
} spc_norm_rope_dims;

/*
 * spc_rope with a norm of each query and key head before the rotation, in the
 * same pass, and with positions of up to four axes: a row x of 128 elements
 * becomes
 *   x_j * w_j / sqrt(mean(x^2) + eps),
 * and pair i of that is turned by pos[axis[i]] * f_i.  Elements rot .. 127 are
 * normed and not turned.
 *   pos      : int32 [axes][B][T] (device).
 *   q_weight : fp32 [128] (device), or NULL: query rows are not normed.
 *   k_weight : the same of the key rows.
 * The values' rows are copied as they are.  Everything else as spc_rope.  The
 * mean, the norm and the rotation are binary32, rounded once to bf16; squares
 * that overflow binary32 are formed of scaled elements.  x_j * w_j is formed
 * before the division: beyond 2^127 it overflows, and below 2^-126 it loses bits
 * (rows whose squares overflow are multiplied by 2^-70 first).
 */
spc_status spc_norm_rope(const spc_norm_rope_dims* d, const int32_t* pos, const uint64_t* turns, const float* q_weight,
                         const float* k_weight, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                         uint16_t* q_out, uint16_t* k_out, uint16_t* v_out, spc_stream stream);

/*
 * Causal attention of prompts over 16-bit keys and values (SpeCache page,
 * section 3 "Prefilling": the attention that Quant and Offload follow).
 * S sequences; sequence s has lq query tokens, the last of its lk tokens, and
 * query i sees keys j <= i + lk - lq:
 *   o_i = sum_j softmax_j(scale * q_i.k_j) v_j,  lse_i the natural log of the
 * normaliser.  Query head h uses KV head h / G, G = Hq / Hkv (1 .. 128).  A
 * query that sees no key (lk < lq) gets o = 0 and lse = -infinity.
 * What keys and values hold in places that a query does not see does not
 * change its output, infinities and NaN included.  The weighted sum of values
 * is formed before it is divided by the sum of weights, with weights of up to
 * 2^8, in binary32: values beyond 2^119 / (number of keys) may overflow in it.
 */
typedef struct spc_prompt_dims {
  int32_t S, Hq, Hkv, D;      /* D = 128 */
  int32_t q_tokens, k_tokens; /* tokens that the token axes of q, o and of k, v hold */
  int32_t q_max, k_max;       /* no sequence has more query tokens / keys than these */
  float scale;
  spc_layout q, k, v, o;      /* b = 0: the sequences lie on one token axis (packed); else sequence s at s * b.
                                 q and o alike, k and v alike */
} spc_prompt_dims;

/* Bytes of device workspace of spc_prompt_attn on the current device: a status
 * word (256 bytes; zero-filled once by the caller for
 * spc_prompt_attn_status) and, where few queries leave SMs idle and the keys
 * are split, the splits' partial results.  256 says that there is no split:
 * the call then also takes ws = NULL.  Calls that
 * share a workspace must not overlap on the GPU.  0 for an invalid shape. */
size_t spc_prompt_attn_workspace_bytes(const spc_prompt_dims* d);

/*
 *   q, k, v : bf16 views; k and v may be NULL when k_max = 0.
 *   q_begin, q_len, k_begin, k_len : int32 [S] (device) or NULL: each
 *            sequence's first token on its token axis (NULL: 0) and its
 *            length (NULL: q_max, k_max).  Values are held to the tensors
 *            (0 .. q_tokens and so on) and to q_max, k_max.  Packed queries
 *            of several sequences need q_begin; sequences may share keys.
 *   o       : bf16, rows of no sequence are left as they were; sequences'
 *            rows must not overlap, and the view shares no byte range with an
 *            input (SPC_ERR_INVALID).
 *   lse     : fp32 [q_tokens][Hq] (packed) or [S][q_tokens][Hq], or NULL.
 *   ws      : at least spc_prompt_attn_workspace_bytes(d) bytes, or NULL with
 *            ws_bytes 0 where that is 256.
 * Neither lse nor those bytes of ws share a byte range with another tensor
 * (SPC_ERR_INVALID).
 * One launch, and a second, small one where the keys are split.
 */
spc_status spc_prompt_attn(const spc_prompt_dims* d, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                           const int32_t* q_begin, const int32_t* q_len, const int32_t* k_begin,
                           const int32_t* k_len, uint16_t* o, float* lse, void* ws, size_t ws_bytes,
                           spc_stream stream);

/* Reads and clears the status word of a workspace of spc_prompt_attn (or
 * spc_window_attn or spc_prefix_attn), or, with ws = NULL, the current device's,
 * which every call on the device reports to as well: SPC_ERR_TIMEOUT if a bounded wait ran out since, else SPC_OK.
 * Synchronises `stream`. */
spc_status spc_prompt_attn_status(void* ws, spc_stream stream);

/* The limit of a wait in the kernels of spc_prompt_attn, spc_window_attn and
 * spc_prefix_attn, in ns (2 * 10^9 unless set;
 * regular waits last microseconds, but for one that lasts as long as a CTA
 * walks over keys that its rows see in full: its limit grows with them).  ns >
 * 0 sets it, to 10^12 at most, for the calls of the process from now on (a
 * captured call keeps the one it was captured with), any other value changes nothing.  Returns the
 * limit before the call.  A wait that runs out ends its CTA early, whose rows
 * of o and lse then hold no result. */
int64_t spc_prompt_attn_wait_limit(int64_t ns);

/*
 * spc_prompt_attn with a sliding window and first tokens that stay visible
 * ("attention sinks"): the query at place p = i + lk - lq of its sequence sees
 * the keys j <= p with j > p - window (its own and the window - 1 before it) or
 * j < sinks.  window >= 1, sinks >= 0; a window of k_max or more leaves
 * spc_prompt_attn, and makes its call.  Keys and values that no query of a call
 * sees are not used (and mostly not read).  Arguments, results, refusals and
 * the workspace's rules are spc_prompt_attn's; spc_prompt_attn_status and
 * spc_prompt_attn_wait_limit cover its waits.
 */
size_t spc_window_attn_workspace_bytes(const spc_prompt_dims* d, int32_t window, int32_t sinks);

spc_status spc_window_attn(const spc_prompt_dims* d, int32_t window, int32_t sinks, const uint16_t* q,
                           const uint16_t* k, const uint16_t* v, const int32_t* q_begin, const int32_t* q_len,
                           const int32_t* k_begin, const int32_t* k_len, uint16_t* o, float* lse, void* ws,
                           size_t ws_bytes, spc_stream stream);

/* A prefix that all sequences of a call share: [tokens][Hkv][D] rows of keys and of values. */
typedef struct spc_prefix {
  int32_t tokens;  /* that the views hold: 0 .. 2^30 - 1 */
  spc_layout k, v; /* (b is not used) */
} spc_prefix;

/*
 * spc_prompt_attn of sequences that share a prefix, stored once: every query
 * sees all P tokens of the prefix, and of its own sequence's lk keys those
 * j <= i + lk - lq.
 *   pk, pv : bf16 views of the prefix's rows; may be NULL when p->tokens = 0,
 *            which leaves spc_prompt_attn, and makes its call.
 *   p_len  : int32 [1] (device) or NULL: P (NULL: p->tokens), held to 0 ..
 *            p->tokens.
 * A query that sees no key of its own sequence has the prefix; k_max may be 0.
 * Everything else as spc_prompt_attn (neither o, lse nor the workspace shares a
 * byte range with the prefix).
 */
size_t spc_prefix_attn_workspace_bytes(const spc_prompt_dims* d, const spc_prefix* p);

/* How a call of this shape on the current device walks over the prefix: once
 * for the rows of all sequences together, with their own keys in the same walk
 * (2) or in a launch of their own (1); or for each sequence by itself (0, and
 * for an invalid shape), where that takes no longer or tiles would hold few
 * rows: batched queries of which no two sequences fit into a tile of 128 G-head
 * rows (2 * q_max > 128 / G), or with a q_begin (placed != 0); packed ones on an
 * axis of more than 4 * S * q_max tokens. */
int32_t spc_prefix_attn_together(const spc_prompt_dims* d, const spc_prefix* p, int32_t placed);

spc_status spc_prefix_attn(const spc_prompt_dims* d, const spc_prefix* p, const uint16_t* q, const uint16_t* pk,
                           const uint16_t* pv, const int32_t* p_len, const uint16_t* k, const uint16_t* v,
                           const int32_t* q_begin, const int32_t* q_len, const int32_t* k_begin,
                           const int32_t* k_len, uint16_t* o, float* lse, void* ws, size_t ws_bytes,
                           spc_stream stream);

/*
 * A run of n new tokens joins the cache (SpeCache page, Algorithm 1 for a
 * prompt: d->N = 0; a follow-up prompt of a conversation: d->N > 0).  The
 * result is bit-identical to n calls of spc_append_kv, and so to
 * spc_quantize_kv over all N + n tokens.  d describes the cache BEFORE the
 * call; the caller then advances d->N by n.
 *   k_new, v_new: bf16 views [B][n][Hkv][D] of the tokens N .. N+n-1 (device).
 *   records, resid: the cache (device), updated in place.
 *   host_kv: HOST pointer to the pinned, mapped cache [B][Hkv][n_cap][2][D]
 *            (rows N .. N+n-1 are written), or NULL for no offload;
 *            SPC_ERR_NOT_MAPPED if not mapped; n_cap >= N + n.
 * Needs q_groups_cap >= N_q'/32 and resid_cap >= N + n - N_q' and the old
 * N - N_q (SPC_ERR_INVALID otherwise), N_q' the quantised tokens of N + n.
 */
spc_status spc_extend_kv(const spc_dims* d, int32_t n, const uint16_t* k_new, const uint16_t* v_new,
                         const spc_layout* k_layout, const spc_layout* v_layout, void* records, uint16_t* resid,
                         uint16_t* host_kv, int64_t n_cap, spc_stream stream);

/*
 * Reads tokens first .. first+n-1 of the cache back as 16-bit rows, for a
 * follow-up prompt's attention over the history: a quantised token's elements
 * are fl(z + fl(s * code)) in binary32 (z and s from the group's min and max
 * as under spc_records_bytes), rounded once to bf16; a residual token's are
 * its 16-bit rows.
 *   k, v: bf16 views [B][n][Hkv][D] (device) that share no row (SPC_ERR_INVALID; views of
 *         different strides that reach into one another are only compared by
 *         their first rows); other rows are left as they were.
 * first >= 0, n >= 0, first + n <= N.
 */
spc_status spc_dequantize_kv(const spc_dims* d, const void* records, const uint16_t* resid, int32_t first, int32_t n,
                             uint16_t* k, uint16_t* v, const spc_layout* k_layout, const spc_layout* v_layout,
                             spc_stream stream);

/*
 * What spc_rope, spc_norm_rope, spc_prompt_attn, spc_window_attn,
 * spc_prefix_attn, spc_extend_kv and spc_dequantize_kv would refuse, without a
 * launch: the same arguments, and the status that the call
 * would return before it enqueues anything.  For a sequence of calls of which
 * either all are to be made or none (a prompt is rotated in place before its
 * attention and its way into the cache).
 */
spc_status spc_rope_check(const spc_rope_dims* d, const int32_t* pos, const uint64_t* turns, const uint16_t* q,
                          const uint16_t* k, const uint16_t* v, uint16_t* q_out, uint16_t* k_out, uint16_t* v_out,
                          spc_stream stream);
spc_status spc_norm_rope_check(const spc_norm_rope_dims* d, const int32_t* pos, const uint64_t* turns,
                               const float* q_weight, const float* k_weight, const uint16_t* q, const uint16_t* k,
                               const uint16_t* v, uint16_t* q_out, uint16_t* k_out, uint16_t* v_out, spc_stream stream);
spc_status spc_prompt_attn_check(const spc_prompt_dims* d, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                 const int32_t* q_begin, const int32_t* q_len, const int32_t* k_begin,
                                 const int32_t* k_len, uint16_t* o, float* lse, void* ws, size_t ws_bytes,
                                 spc_stream stream);
spc_status spc_window_attn_check(const spc_prompt_dims* d, int32_t window, int32_t sinks, const uint16_t* q,
                                 const uint16_t* k, const uint16_t* v, const int32_t* q_begin, const int32_t* q_len,
                                 const int32_t* k_begin, const int32_t* k_len, uint16_t* o, float* lse, void* ws,
                                 size_t ws_bytes, spc_stream stream);
spc_status spc_prefix_attn_check(const spc_prompt_dims* d, const spc_prefix* p, const uint16_t* q, const uint16_t* pk,
                                 const uint16_t* pv, const int32_t* p_len, const uint16_t* k, const uint16_t* v,
                                 const int32_t* q_begin, const int32_t* q_len, const int32_t* k_begin,
                                 const int32_t* k_len, uint16_t* o, float* lse, void* ws, size_t ws_bytes,
                                 spc_stream stream);
spc_status spc_extend_kv_check(const spc_dims* d, int32_t n, const uint16_t* k_new, const uint16_t* v_new,
                               const spc_layout* k_layout, const spc_layout* v_layout, void* records, uint16_t* resid,
                               uint16_t* host_kv, int64_t n_cap, spc_stream stream);
spc_status spc_dequantize_kv_check(const spc_dims* d, const void* records, const uint16_t* resid, int32_t first,
                                   int32_t n, uint16_t* k, uint16_t* v, const spc_layout* k_layout,
                                   const spc_layout* v_layout, spc_stream stream);

/*
 * Decode-time append (SpeCache page, section 3 "Decoding", Algorithm 3: the
 * new token's K/V joins the cache; section 3: the full-precision cache is
 * offloaded to CPU memory).  d describes the cache BEFORE the call: N tokens
 * held as records + resid, as spc_quantize_kv (or earlier appends) left them.
 * Afterwards the cache holds N+1 tokens and the caller advances d->N.
 *   k_new, v_new: bf16 [B][Hkv][D], token N's key and value rows (device).
 *   records, resid: the cache (device), updated in place.
 *   host_kv: HOST pointer to the pinned, mapped full-precision cache
 *            [B][Hkv][n_cap][2][D] (row N is written), or NULL for no
 *            offload; SPC_ERR_NOT_MAPPED if not mapped; n_cap > N.
 * The new row goes to window row r = N - N_q.  When N+1 tokens quantise one
 * more group (N_q' = N_q + g), the window's oldest g rows are quantised
 * into record N_q/g and the window shifts down by g rows; the result is
 * bit-identical to spc_quantize_kv over all N+1 tokens.  Needs
 * resid_cap >= N - N_q + 1 and, at a flush, q_groups_cap >= N_q'/32
 * (SPC_ERR_INVALID otherwise).  One launch on `stream`.
 */
spc_status spc_append_kv(const spc_dims* d, const uint16_t* k_new, const uint16_t* v_new, void* records,
                         uint16_t* resid, uint16_t* host_kv, int64_t n_cap, spc_stream stream);

/*
 * ArgTopK(A_{1,:}) (Algorithm 3): per (b, hkv), the k_eff = min(k, N_q)
 * quantised positions n with the largest score
 *   S(n) = sum over the G query heads h of KV head hkv of
 *          exp(spec_logits[b][hkv][h%G][n] - lse[b][1][h]),
 * i.e. the speculative token's attention probability summed over the group.
 * Ties go to the lower position.  Outputs: idx int32 [B][Hkv][k], ascending,
 * entries k_eff..k-1 set to -1; bitmap u32 [B][Hkv][q_groups_cap] with
 * exactly the selected bits set (words past N_q/32 are zeroed).
 * N_q <= 262144; spec_logits 16-byte aligned (SPC_ERR_INVALID otherwise).
 */
spc_status spc_topk_select(const spc_dims* d, const float* spec_logits, const float* lse,
                           int32_t k, int32_t* idx, uint32_t* bitmap, spc_stream stream);

/*
 * spc_topk_select that also says where each selected position sat in the
 * previous selection, so that a pre-fetch copies only the rows it does not
 * hold yet (spc_merged_attn_fetch_prev):
 *   prev_idx: int32 [B][Hkv][prev_k], the previous selection (ascending,
 *             -1 padded at the end, as spc_topk_select writes it); may be NULL
 *             when prev_k = 0.
 *   src:      int32 [B][Hkv][k] output: src[b][hkv][j] = the index i with
 *             prev_idx[b][hkv][i] == idx[b][hkv][j], else -1 (also for the
 *             -1 entries j >= k_eff).
 * idx and bitmap are exactly spc_topk_select's.  prev_idx must not share a
 * byte with idx (SPC_ERR_INVALID).
 */
spc_status spc_topk_select_prev(const spc_dims* d, const float* spec_logits, const float* lse,
                                int32_t k, int32_t* idx, uint32_t* bitmap, const int32_t* prev_idx,
                                int32_t prev_k, int32_t* src, spc_stream stream);

/*
 * Pre-fetch(C_kappa) (Algorithm 3): copies the selected 16-bit rows from the
 * full-precision cache in CPU memory into HBM,
 *   staging[b][hkv][j][t][:] = host_kv[b][hkv][idx[b][hkv][j]][t][:], t in {K, V},
 * for j < k with idx >= 0 (other staging rows are left untouched).
 *   host_kv : HOST pointer, bf16 [B][Hkv][n_cap][2][D], pinned and mapped
 *             into the device address space (cudaHostAlloc / cudaHostRegister
 *             with mapping); otherwise SPC_ERR_NOT_MAPPED.
 *   max_ctas: bound on the copy kernel's grid (0 = library default), so the
 *             copy can share the GPU with attention running on another stream.
 * Indices must be < n_cap.  The copy is issued on `stream`, typically a side
 * stream ordered after spc_topk_select by an event.
 */
spc_status spc_host_gather(const spc_dims* d, const uint16_t* host_kv, int64_t n_cap,
                           const int32_t* idx, int32_t k, uint16_t* staging, int32_t max_ctas,
                           spc_stream stream);

/*
 * spc_host_gather that keeps the rows already staged (SpeCache page, section
 * 3: the used 16-bit rows outside the new top-k are evicted, the others
 * stay): row j with src[b][hkv][j] >= 0 is copied from
 * prev_staging[b][hkv][src[b][hkv][j]] (device, [B][Hkv][prev_k][2][D]), the
 * others from the host cache.  src is what spc_topk_select_prev writes for
 * idx against the previous selection, whose rows prev_staging holds; staging
 * is then exactly spc_host_gather's.  prev_staging must not share a byte
 * with staging (SPC_ERR_INVALID; 16-byte aligned; NULL only with prev_k = 0).  Everything else as
 * spc_host_gather.
 */
spc_status spc_host_gather_prev(const spc_dims* d, const uint16_t* host_kv, int64_t n_cap,
                                const int32_t* idx, int32_t k, uint16_t* staging, const int32_t* src,
                                const uint16_t* prev_staging, int32_t prev_k, int32_t max_ctas,
                                spc_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* SPC_H */
