// extern "C" entry points of libspc (declared in include/spc.h): argument
// validation, then one launch sequence per call on the caller's stream.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "common.cuh"

namespace spc {
spc_status launch_quantize(const spc_dims*, const uint16_t*, const uint16_t*, void*, uint16_t*, cudaStream_t);
size_t attn_workspace_bytes(const spc_dims*, int32_t);
spc_status launch_attention(const spc_dims*, const void*, const uint16_t*, const uint16_t*, const uint16_t*,
                            const int32_t*, const uint32_t*, const uint16_t*, int32_t, uint16_t*, float*, float*,
                            void*, cudaStream_t, const PrefetchJob*, const SelectJob*, bool*);
size_t step_workspace_bytes(const spc_dims*, int32_t);
int attn_kernel_count(const spc_dims*, int32_t, int32_t);
int step_kernel_count(const spc_dims*, int32_t, int32_t, int32_t);
bool step_onchip(const spc_dims*, int32_t, int32_t, int32_t);
spc_status launch_topk(const spc_dims*, const float*, const float*, int32_t, int32_t*, uint32_t*, cudaStream_t,
                       const int32_t* prev_idx = nullptr, int32_t prev_k = 0, int32_t* src = nullptr);
spc_status launch_host_gather(const spc_dims*, const uint16_t*, int64_t, const int32_t*, int32_t, uint16_t*,
                              int32_t, cudaStream_t, const int32_t* src = nullptr, const uint16_t* prev = nullptr,
                              int32_t prev_k = 0);
spc_status launch_append(const spc_dims*, const uint16_t*, const uint16_t*, void*, uint16_t*, uint16_t*, int64_t,
                         cudaStream_t);
spc_status launch_rope(const spc_rope_dims*, const int32_t*, const uint64_t*, const uint16_t*, const uint16_t*,
                       const uint16_t*, uint16_t*, uint16_t*, uint16_t*, cudaStream_t);
spc_status launch_norm_rope(const spc_norm_rope_dims*, const int32_t*, const uint64_t*, const float*, const float*,
                            const uint16_t*, const uint16_t*, const uint16_t*, uint16_t*, uint16_t*, uint16_t*,
                            cudaStream_t);
size_t prompt_workspace_bytes(const spc_prompt_dims*);
size_t window_workspace_bytes(const spc_prompt_dims*, int32_t, int32_t);
size_t prefix_workspace_bytes(const spc_prompt_dims*, const spc_prefix*);
int32_t prefix_together(const spc_prompt_dims*, const spc_prefix*, bool);
cudaError_t window_fault_word(void**);
cudaError_t prefix_fault_word(void**);
spc_status launch_window_attn(const spc_prompt_dims*, int32_t, int32_t, const uint16_t*, const uint16_t*,
                              const uint16_t*, const int32_t*, const int32_t*, const int32_t*, const int32_t*,
                              uint16_t*, float*, void*, cudaStream_t);
spc_status launch_prefix_attn(const spc_prompt_dims*, const spc_prefix*, const uint16_t*, const uint16_t*,
                              const uint16_t*, const int32_t*, const uint16_t*, const uint16_t*, const int32_t*,
                              const int32_t*, const int32_t*, const int32_t*, uint16_t*, float*, void*, cudaStream_t);
int64_t prompt_wait_limit(int64_t);
cudaError_t prompt_fault_word(void**);
spc_status launch_prompt_attn(const spc_prompt_dims*, const uint16_t*, const uint16_t*, const uint16_t*,
                              const int32_t*, const int32_t*, const int32_t*, const int32_t*, uint16_t*, float*,
                              void*, cudaStream_t);
spc_status launch_extend(const spc_dims*, int32_t, const uint16_t*, const uint16_t*, const spc_layout*,
                         const spc_layout*, void*, uint16_t*, uint16_t*, int64_t, cudaStream_t);
spc_status launch_dequantize(const spc_dims*, const void*, const uint16_t*, int32_t, int32_t, uint16_t*, uint16_t*,
                             const spc_layout*, const spc_layout*, cudaStream_t);
}  // namespace spc

namespace spc_host {

static thread_local int32_t g_last_cuda_error = 0;

void set_cuda_error(cudaError_t e) { g_last_cuda_error = (int32_t)e; }

int sm_count() {
  static std::mutex mu;
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  std::lock_guard<std::mutex> lock(mu);
  if (cached[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    cached[dev] = n;
  }
  return cached[dev];
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int current_device() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  return dev;
}

}  // namespace spc_host

namespace {

using spc_host::aligned16;

// Shape checks shared by every call.
spc_status check_dims(const spc_dims* d) {
  if (d == nullptr) return SPC_ERR_INVALID;
  if (d->B <= 0 || d->Hq <= 0 || d->Hkv <= 0 || d->D <= 0 || d->N < 0 || d->R < 0 || d->q_groups_cap < 0 ||
      d->resid_cap < 0)
    return SPC_ERR_INVALID;
  if (d->Hq % d->Hkv != 0) return SPC_ERR_INVALID;
  if (d->bits != 1 && d->bits != 2) return SPC_ERR_INVALID;
  if (!(std::isfinite(d->scale) && d->scale > 0.f)) return SPC_ERR_INVALID;
  const int G = d->Hq / d->Hkv;
  if (d->D != spc::kD || (d->group != 32 && d->group != 64)) return SPC_ERR_UNSUPPORTED;
  if (G != 1 && G != 2 && G != 4) return SPC_ERR_UNSUPPORTED;
  const int32_t nq = spc::num_quantized(d->N, d->R, d->group);
  if (nq / spc::kGroup > d->q_groups_cap) return SPC_ERR_INVALID;
  if (d->N - nq > d->resid_cap) return SPC_ERR_INVALID;
  return SPC_OK;
}

// Device address of a pinned, mapped host buffer, or SPC_ERR_NOT_MAPPED.
spc_status mapped_device_pointer(const void* host, const void** dev) {
  cudaPointerAttributes attr;
  const cudaError_t e = cudaPointerGetAttributes(&attr, host);
  if (e != cudaSuccess) {
    cudaGetLastError();  // the failed query leaves no sticky error; clear it
    return SPC_ERR_NOT_MAPPED;
  }
  if (attr.type != cudaMemoryTypeHost || attr.devicePointer == nullptr) return SPC_ERR_NOT_MAPPED;
  *dev = attr.devicePointer;
  return SPC_OK;
}

}  // namespace

namespace spc_host {

// Argument checks of every attention entry point other than those of its
// workspace, in the order they apply; nothing is launched or enqueued.
spc_status check_attn_args(const spc_dims* d, const void* records, const uint16_t* resid, const uint16_t* q,
                           const uint16_t* kv_self, const int32_t* idx, const uint32_t* bitmap,
                           const uint16_t* staging, int32_t k, const uint16_t* o, const float* lse,
                           const float* spec_logits) {
  spc_status st = check_dims(d);
  if (st != SPC_OK) return st;
  const int32_t nq = spc::num_quantized(d->N, d->R, d->group);
  if (q == nullptr || o == nullptr) return SPC_ERR_INVALID;
  if (nq > 0 && records == nullptr) return SPC_ERR_INVALID;
  if (d->N - nq > 0 && resid == nullptr) return SPC_ERR_INVALID;
  if (!aligned16(records) || !aligned16(resid) || !aligned16(q) || !aligned16(kv_self) || !aligned16(o) ||
      !aligned16(lse) || !aligned16(spec_logits))
    return SPC_ERR_INVALID;
  if (k < 0 || k > (1 << 24)) return SPC_ERR_INVALID;
  if (k > 0) {
    if (idx == nullptr || bitmap == nullptr || staging == nullptr || !aligned16(staging)) return SPC_ERR_INVALID;
  }
  return SPC_OK;
}

}  // namespace spc_host

namespace {

// [a, a + na) and [b, b + nb) share a byte
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (a == nullptr || b == nullptr || na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}
// bytes of a [B][Hkv][k][2][D] bf16 staging buffer
size_t staging_bytes(const spc_dims* d, int64_t k) { return (size_t)d->B * d->Hkv * (size_t)k * 2 * d->D * 2; }
// A carried pre-fetch writes fetch_staging while the attention reads staging
// (k rows) and, with kept rows, copies from prev (prev_k rows): a shared byte
// would race.
bool fetch_buffers_overlap(const spc_dims* d, const uint16_t* staging, int32_t k, const uint16_t* fetch_staging,
                           int32_t fetch_k, const uint16_t* prev, int32_t prev_k) {
  const size_t out = staging_bytes(d, fetch_k);
  return (k > 0 && overlap(staging, staging_bytes(d, k), fetch_staging, out)) ||
         (prev_k > 0 && overlap(prev, staging_bytes(d, prev_k), fetch_staging, out));
}

spc_status attn_common(const spc_dims* d, const void* records, const uint16_t* resid, const uint16_t* q,
                       const uint16_t* kv_self, const int32_t* idx, const uint32_t* bitmap, const uint16_t* staging, int32_t k,
                       uint16_t* o, float* lse, float* spec_logits, void* ws, size_t ws_bytes,
                       spc_stream stream, const spc::PrefetchJob* pf = nullptr,
                       const spc::SelectJob* sel = nullptr, bool* sel_done = nullptr) {
  spc_status st = spc_host::check_attn_args(d, records, resid, q, kv_self, idx, bitmap, staging, k, o, lse,
                                            spec_logits);
  if (st != SPC_OK) return st;
  if (ws == nullptr || !aligned16(ws)) return SPC_ERR_INVALID;
  const size_t need = sel != nullptr ? spc::step_workspace_bytes(d, std::max(k, sel->k))
                                     : spc::attn_workspace_bytes(d, k);
  if (ws_bytes < need) return SPC_ERR_WORKSPACE;
  return spc::launch_attention(d, records, resid, q, kv_self, k > 0 ? idx : nullptr, k > 0 ? bitmap : nullptr,
                               k > 0 ? staging : nullptr, k, o, lse, spec_logits, ws,
                               reinterpret_cast<cudaStream_t>(stream), pf, sel, sel_done);
}

}  // namespace

extern "C" {

int32_t spc_abi_version(void) { return SPC_ABI_VERSION; }

const char* spc_status_string(spc_status s) {
  switch (s) {
    case SPC_OK: return "ok";
    case SPC_ERR_INVALID: return "invalid argument";
    case SPC_ERR_UNSUPPORTED: return "unsupported shape";
    case SPC_ERR_CUDA: return "CUDA error";
    case SPC_ERR_NOT_MAPPED: return "host pointer is not mapped pinned memory";
    case SPC_ERR_WORKSPACE: return "workspace too small";
    case SPC_ERR_TIMEOUT: return "a kernel's bounded wait ran out (see spc_read_device_status)";
  }
  return "unknown status";
}

int32_t spc_last_cuda_error(void) { return spc_host::g_last_cuda_error; }

int32_t spc_num_quantized(const spc_dims* d) {
  if (check_dims(d) == SPC_ERR_INVALID) return -1;
  return spc::num_quantized(d->N, d->R, d->group);
}

size_t spc_records_bytes(const spc_dims* d) {
  if (d == nullptr || d->B <= 0 || d->Hkv <= 0 || d->q_groups_cap < 0 || (d->bits != 1 && d->bits != 2) ||
      (d->group != 32 && d->group != 64))
    return 0;
  return (size_t)d->B * d->Hkv * spc::records_cap(d->group, d->q_groups_cap) *
         (size_t)spc::record_bytes(d->bits, d->group);
}

size_t spc_resid_bytes(const spc_dims* d) {
  if (d == nullptr || d->B <= 0 || d->Hkv <= 0 || d->resid_cap < 0 || d->D <= 0) return 0;
  return (size_t)d->B * d->Hkv * d->resid_cap * 2 * d->D * sizeof(uint16_t);
}

spc_status spc_quantize_kv(const spc_dims* d, const uint16_t* k, const uint16_t* v, void* records,
                           uint16_t* resid, spc_stream stream) {
  spc_status st = check_dims(d);
  if (st != SPC_OK) return st;
  const int32_t nq = spc::num_quantized(d->N, d->R, d->group);
  if (d->N > 0 && (k == nullptr || v == nullptr)) return SPC_ERR_INVALID;
  if (nq > 0 && records == nullptr) return SPC_ERR_INVALID;
  if (d->N - nq > 0 && resid == nullptr) return SPC_ERR_INVALID;
  if (!aligned16(k) || !aligned16(v) || !aligned16(records) || !aligned16(resid)) return SPC_ERR_INVALID;
  return spc::launch_quantize(d, k, v, records, resid, reinterpret_cast<cudaStream_t>(stream));
}

spc_status spc_offload_kv(const spc_dims* d, const uint16_t* k, const uint16_t* v, uint16_t* host_kv,
                          int64_t n_cap, spc_stream stream) {
  spc_status st = check_dims(d);
  if (st != SPC_OK) return st;
  if (d->N == 0) return SPC_OK;
  if (k == nullptr || v == nullptr || host_kv == nullptr || n_cap < d->N) return SPC_ERR_INVALID;
  if (!aligned16(k) || !aligned16(v) || !aligned16(host_kv)) return SPC_ERR_INVALID;
  const void* host_dev = nullptr;
  st = mapped_device_pointer(host_kv, &host_dev);  // pinned host memory: the copy engines reach it directly
  if (st != SPC_OK) return st;
  const size_t row = (size_t)spc::kD * sizeof(uint16_t);  // 256 bytes
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // rows (b, hkv, n) of K go to host rows (b, hkv, n) at byte 0, of V at byte 256:
  // one strided copy of all B*Hkv*N rows when n_cap == N, else one per (b, hkv)
  // run of N rows (the host runs are n_cap rows apart)
  const int64_t BH = (int64_t)d->B * d->Hkv;
  const int64_t runs = n_cap == d->N ? 1 : BH;
  const size_t height = (size_t)(n_cap == d->N ? BH * d->N : d->N);
  for (int64_t bh = 0; bh < runs; ++bh) {
    for (int kv = 0; kv < 2; ++kv) {
      const uint16_t* src = (kv == 0 ? k : v) + bh * (int64_t)d->N * spc::kD;
      uint16_t* dst = host_kv + (bh * n_cap * 2 + kv) * spc::kD;
      const cudaError_t e = cudaMemcpy2DAsync(dst, 2 * row, src, row, row, height, cudaMemcpyDeviceToHost, s);
      if (e != cudaSuccess) {
        spc_host::set_cuda_error(e);
        return SPC_ERR_CUDA;
      }
    }
  }
  return SPC_OK;
}

spc_status spc_append_kv(const spc_dims* d, const uint16_t* k_new, const uint16_t* v_new, void* records,
                         uint16_t* resid, uint16_t* host_kv, int64_t n_cap, spc_stream stream) {
  spc_status st = check_dims(d);
  if (st != SPC_OK) return st;
  if (d->N >= (1 << 30)) return SPC_ERR_INVALID;
  const int32_t nq = spc::num_quantized(d->N, d->R, d->group);
  const int32_t nq1 = spc::num_quantized(d->N + 1, d->R, d->group);
  if (k_new == nullptr || v_new == nullptr || resid == nullptr) return SPC_ERR_INVALID;
  if (d->N - nq + 1 > d->resid_cap) return SPC_ERR_INVALID;  // room for the new row
  if (nq1 > nq && (records == nullptr || nq1 / spc::kGroup > d->q_groups_cap)) return SPC_ERR_INVALID;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(records) || !aligned16(resid) || !aligned16(host_kv))
    return SPC_ERR_INVALID;
  const void* host_dev = nullptr;
  if (host_kv != nullptr) {
    if (n_cap <= d->N) return SPC_ERR_INVALID;
    st = mapped_device_pointer(host_kv, &host_dev);
    if (st != SPC_OK) return st;
  }
  return spc::launch_append(d, k_new, v_new, records, resid, static_cast<uint16_t*>(const_cast<void*>(host_dev)),
                            n_cap, reinterpret_cast<cudaStream_t>(stream));
}

size_t spc_attn_workspace_bytes(const spc_dims* d, int32_t k_max) {
  if (check_dims(d) != SPC_OK || k_max < 0 || k_max > (1 << 24)) return 0;
  return spc::attn_workspace_bytes(d, k_max);
}

spc_status spc_decode_attn2(const spc_dims* d, const void* records, const uint16_t* resid, const uint16_t* q,
                            const uint16_t* kv_self, uint16_t* o, float* lse, float* spec_logits, void* ws,
                            size_t ws_bytes, spc_stream stream) {
  return attn_common(d, records, resid, q, kv_self, nullptr, nullptr, nullptr, 0, o, lse, spec_logits, ws,
                     ws_bytes, stream);
}

spc_status spc_merged_attn(const spc_dims* d, const void* records, const uint16_t* resid, const uint16_t* q,
                           const uint16_t* kv_self, const int32_t* idx, const uint32_t* bitmap,
                           const uint16_t* staging, int32_t k, uint16_t* o, float* lse, float* spec_logits,
                           void* ws, size_t ws_bytes, spc_stream stream) {
  return attn_common(d, records, resid, q, kv_self, idx, bitmap, staging, k, o, lse, spec_logits, ws, ws_bytes,
                     stream);
}

spc_status spc_merged_attn_fetch(const spc_dims* d, const void* records, const uint16_t* resid,
                                 const uint16_t* q, const uint16_t* kv_self, const int32_t* idx, const uint32_t* bitmap,
                                 const uint16_t* staging, int32_t k, uint16_t* o, float* lse, float* spec_logits,
                                 void* ws, size_t ws_bytes, const uint16_t* fetch_host_kv, int64_t fetch_n_cap,
                                 const int32_t* fetch_idx, int32_t fetch_k, uint16_t* fetch_staging,
                                 spc_stream stream) {
  spc_status st = check_dims(d);
  if (st != SPC_OK) return st;
  if (fetch_k < 0 || fetch_k > (1 << 24) || fetch_n_cap < 0) return SPC_ERR_INVALID;
  if (fetch_k == 0)
    return attn_common(d, records, resid, q, kv_self, idx, bitmap, staging, k, o, lse, spec_logits, ws, ws_bytes,
                       stream);
  if (fetch_host_kv == nullptr || fetch_idx == nullptr || fetch_staging == nullptr) return SPC_ERR_INVALID;
  if (!aligned16(fetch_host_kv) || !aligned16(fetch_staging)) return SPC_ERR_INVALID;
  if (fetch_buffers_overlap(d, staging, k, fetch_staging, fetch_k, nullptr, 0)) return SPC_ERR_INVALID;
  const void* dev = nullptr;
  st = mapped_device_pointer(fetch_host_kv, &dev);
  if (st != SPC_OK) return st;
  spc::PrefetchJob job{static_cast<const uint16_t*>(dev), fetch_n_cap, fetch_idx, fetch_k, fetch_staging};
  return attn_common(d, records, resid, q, kv_self, idx, bitmap, staging, k, o, lse, spec_logits, ws, ws_bytes,
                     stream, &job);
}

spc_status spc_merged_attn_fetch_prev(const spc_dims* d, const void* records, const uint16_t* resid,
                                      const uint16_t* q, const uint16_t* kv_self, const int32_t* idx,
                                      const uint32_t* bitmap, const uint16_t* staging, int32_t k, uint16_t* o,
                                      float* lse, float* spec_logits, void* ws, size_t ws_bytes,
                                      const uint16_t* fetch_host_kv, int64_t fetch_n_cap, const int32_t* fetch_idx,
                                      int32_t fetch_k, uint16_t* fetch_staging, const int32_t* fetch_src,
                                      const uint16_t* fetch_prev_staging, int32_t fetch_prev_k, spc_stream stream) {
  spc_status st = check_dims(d);
  if (st != SPC_OK) return st;
  if (fetch_k < 0 || fetch_k > (1 << 24) || fetch_n_cap < 0 || fetch_prev_k < 0 || fetch_prev_k > (1 << 24))
    return SPC_ERR_INVALID;
  if (fetch_k == 0)
    return attn_common(d, records, resid, q, kv_self, idx, bitmap, staging, k, o, lse, spec_logits, ws, ws_bytes,
                       stream);
  if (fetch_host_kv == nullptr || fetch_idx == nullptr || fetch_staging == nullptr || fetch_src == nullptr)
    return SPC_ERR_INVALID;
  if (!aligned16(fetch_host_kv) || !aligned16(fetch_staging)) return SPC_ERR_INVALID;
  if (fetch_prev_k > 0 && (fetch_prev_staging == nullptr || !aligned16(fetch_prev_staging)))
    return SPC_ERR_INVALID;
  if (fetch_buffers_overlap(d, staging, k, fetch_staging, fetch_k, fetch_prev_staging, fetch_prev_k))
    return SPC_ERR_INVALID;
  const void* dev = nullptr;
  st = mapped_device_pointer(fetch_host_kv, &dev);
  if (st != SPC_OK) return st;
  spc::PrefetchJob job{static_cast<const uint16_t*>(dev), fetch_n_cap, fetch_idx, fetch_k, fetch_staging,
                       fetch_src, fetch_prev_k > 0 ? fetch_prev_staging : nullptr, fetch_prev_k};
  return attn_common(d, records, resid, q, kv_self, idx, bitmap, staging, k, o, lse, spec_logits, ws, ws_bytes,
                     stream, &job);
}

int32_t spc_attn_kernel_count(const spc_dims* d, int32_t k, int32_t fetch_k) {
  if (check_dims(d) != SPC_OK || k < 0 || k > (1 << 24) || fetch_k < 0 || fetch_k > (1 << 24)) return -1;
  return spc::attn_kernel_count(d, k, fetch_k);
}

int32_t spc_decode_step_kernel_count(const spc_dims* d, int32_t k, int32_t fetch_k, int32_t next_k) {
  if (check_dims(d) != SPC_OK || k < 0 || k > (1 << 24) || fetch_k < 0 || fetch_k > (1 << 24) || next_k < 0 ||
      next_k > (1 << 24))
    return -1;
  return spc::step_kernel_count(d, k, fetch_k, next_k);
}

int32_t spc_decode_step_on_chip(const spc_dims* d, int32_t k, int32_t fetch_k, int32_t next_k) {
  if (check_dims(d) != SPC_OK || k < 0 || k > (1 << 24) || fetch_k < 0 || fetch_k > (1 << 24) || next_k < 0 ||
      next_k > (1 << 24))
    return -1;
  return spc::step_onchip(d, k, fetch_k, next_k) ? 1 : 0;
}

size_t spc_step_workspace_bytes(const spc_dims* d, int32_t k_max) {
  if (check_dims(d) != SPC_OK || k_max < 0 || k_max > (1 << 24)) return 0;
  return spc::step_workspace_bytes(d, k_max);
}

// spc_decode_step and spc_decode_step_prev: with next_src, the pre-fetch keeps
// the rows already staged (fetch_src, fetch_prev) and the selection reports
// each position's index in idx.
static spc_status decode_step(const spc_dims* d, const void* records, const uint16_t* resid, const uint16_t* q,
                              const uint16_t* kv_self, const int32_t* idx, const uint32_t* bitmap,
                              const uint16_t* staging, int32_t k, uint16_t* o, float* lse, float* spec_logits,
                              int32_t next_k, int32_t* next_idx, uint32_t* next_bitmap, int32_t* next_src, void* ws,
                              size_t ws_bytes, const uint16_t* fetch_host_kv, int64_t fetch_n_cap,
                              const int32_t* fetch_idx, int32_t fetch_k, uint16_t* fetch_staging,
                              const int32_t* fetch_src, const uint16_t* fetch_prev, int32_t fetch_prev_k,
                              bool keep, spc_stream stream) {
  spc_status st = check_dims(d);
  if (st != SPC_OK) return st;
  const int32_t nq = spc::num_quantized(d->N, d->R, d->group);
  if (next_k < 0 || next_k > (1 << 24)) return SPC_ERR_INVALID;
  if (next_bitmap == nullptr || (next_k > 0 && next_idx == nullptr)) return SPC_ERR_INVALID;
  if (keep && next_k > 0 &&
      (next_src == nullptr || (k > 0 && overlap(next_idx, (size_t)d->B * d->Hkv * next_k * 4, idx,
                                                  (size_t)d->B * d->Hkv * k * 4))))
    return SPC_ERR_INVALID;
  if (nq > 0 && lse == nullptr) return SPC_ERR_INVALID;
  if (nq > 262144) return SPC_ERR_UNSUPPORTED;
  // without a logits buffer the selection must ride on the attention with the logits on chip
  if (nq > 0 && spec_logits == nullptr &&
      (fetch_k < 0 || fetch_k > (1 << 24) || k < 0 || k > (1 << 24) || !spc::step_onchip(d, k, fetch_k, next_k)))
    return SPC_ERR_UNSUPPORTED;
  spc::PrefetchJob job{nullptr, fetch_n_cap, fetch_idx, fetch_k, fetch_staging};
  const spc::PrefetchJob* pf = nullptr;
  if (fetch_k != 0) {
    if (fetch_k < 0 || fetch_k > (1 << 24) || fetch_n_cap < 0) return SPC_ERR_INVALID;
    if (fetch_host_kv == nullptr || fetch_idx == nullptr || fetch_staging == nullptr) return SPC_ERR_INVALID;
    if (!aligned16(fetch_host_kv) || !aligned16(fetch_staging)) return SPC_ERR_INVALID;
    if (keep) {
      if (fetch_src == nullptr || fetch_prev_k < 0 || fetch_prev_k > (1 << 24)) return SPC_ERR_INVALID;
      if (fetch_prev_k > 0 && (fetch_prev == nullptr || !aligned16(fetch_prev))) return SPC_ERR_INVALID;
      job.src = fetch_src;
      job.prev = fetch_prev_k > 0 ? fetch_prev : nullptr;
      job.prev_k = fetch_prev_k;
    }
    if (fetch_buffers_overlap(d, staging, k, fetch_staging, fetch_k, job.prev, job.prev_k)) return SPC_ERR_INVALID;
    const void* dev = nullptr;
    st = mapped_device_pointer(fetch_host_kv, &dev);
    if (st != SPC_OK) return st;
    job.host_dev = static_cast<const uint16_t*>(dev);
    pf = &job;
  }
  spc::SelectJob sel{next_idx, next_bitmap, next_k, keep && next_k > 0 ? next_src : nullptr};
  bool fused = false;
  st = attn_common(d, records, resid, q, kv_self, idx, bitmap, staging, k, o, lse, spec_logits, ws, ws_bytes,
                   stream, pf, &sel, &fused);
  if (st != SPC_OK || fused) return st;
  // the selection could not ride on this attention launch: its own launch, right after
  if (d->q_groups_cap == 0 && next_k == 0) return SPC_OK;
  return spc::launch_topk(d, spec_logits, lse, next_k, next_idx, next_bitmap, reinterpret_cast<cudaStream_t>(stream),
                          idx, k, keep && next_k > 0 ? next_src : nullptr);
}

spc_status spc_decode_step(const spc_dims* d, const void* records, const uint16_t* resid, const uint16_t* q,
                           const uint16_t* kv_self, const int32_t* idx, const uint32_t* bitmap, const uint16_t* staging, int32_t k,
                           uint16_t* o, float* lse, float* spec_logits, int32_t next_k, int32_t* next_idx,
                           uint32_t* next_bitmap, void* ws, size_t ws_bytes, const uint16_t* fetch_host_kv,
                           int64_t fetch_n_cap, const int32_t* fetch_idx, int32_t fetch_k,
                           uint16_t* fetch_staging, spc_stream stream) {
  return decode_step(d, records, resid, q, kv_self, idx, bitmap, staging, k, o, lse, spec_logits, next_k, next_idx,
                     next_bitmap, nullptr, ws, ws_bytes, fetch_host_kv, fetch_n_cap, fetch_idx, fetch_k,
                     fetch_staging, nullptr, nullptr, 0, false, stream);
}

spc_status spc_decode_step_prev(const spc_dims* d, const void* records, const uint16_t* resid, const uint16_t* q,
                                const uint16_t* kv_self, const int32_t* idx, const uint32_t* bitmap,
                                const uint16_t* staging, int32_t k, uint16_t* o, float* lse, float* spec_logits,
                                int32_t next_k, int32_t* next_idx, uint32_t* next_bitmap, int32_t* next_src,
                                void* ws, size_t ws_bytes, const uint16_t* fetch_host_kv, int64_t fetch_n_cap,
                                const int32_t* fetch_idx, int32_t fetch_k, uint16_t* fetch_staging,
                                const int32_t* fetch_src, const uint16_t* fetch_prev_staging, int32_t fetch_prev_k,
                                spc_stream stream) {
  return decode_step(d, records, resid, q, kv_self, idx, bitmap, staging, k, o, lse, spec_logits, next_k, next_idx,
                     next_bitmap, next_src, ws, ws_bytes, fetch_host_kv, fetch_n_cap, fetch_idx, fetch_k,
                     fetch_staging, fetch_src, fetch_prev_staging, fetch_prev_k, true, stream);
}

spc_status spc_read_device_status(void* ws, const spc_dims* d, spc_stream stream) {
  spc_status st = check_dims(d);
  if (st != SPC_OK) return st;
  if (ws == nullptr) return SPC_ERR_INVALID;
  uint32_t* fault = static_cast<uint32_t*>(ws) + 3 * (int64_t)d->B * d->Hkv;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, fault, sizeof(v), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && v != 0u) e = cudaMemsetAsync(fault, 0, sizeof(v), s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) {
    spc_host::set_cuda_error(e);
    return SPC_ERR_CUDA;
  }
  return v != 0u ? SPC_ERR_TIMEOUT : SPC_OK;
}

// The arguments of both top-k entry points; SPC_OK when they are valid.
static spc_status check_topk_args(const spc_dims* d, const float* spec_logits, const float* lse, int32_t k,
                                  const int32_t* idx, const uint32_t* bitmap) {
  spc_status st = check_dims(d);
  if (st != SPC_OK) return st;
  const int32_t nq = spc::num_quantized(d->N, d->R, d->group);
  if (k < 0 || k > (1 << 24)) return SPC_ERR_INVALID;
  if (bitmap == nullptr || (k > 0 && idx == nullptr)) return SPC_ERR_INVALID;
  if (nq > 0 && (spec_logits == nullptr || lse == nullptr)) return SPC_ERR_INVALID;
  if (nq > 0 && !aligned16(spec_logits)) return SPC_ERR_INVALID;  // read in 16-byte pieces
  if (nq > 262144) return SPC_ERR_UNSUPPORTED;
  return SPC_OK;
}

spc_status spc_topk_select(const spc_dims* d, const float* spec_logits, const float* lse, int32_t k,
                           int32_t* idx, uint32_t* bitmap, spc_stream stream) {
  const spc_status st = check_topk_args(d, spec_logits, lse, k, idx, bitmap);
  if (st != SPC_OK) return st;
  if (d->q_groups_cap == 0 && k == 0) return SPC_OK;
  return spc::launch_topk(d, spec_logits, lse, k, idx, bitmap, reinterpret_cast<cudaStream_t>(stream));
}

spc_status spc_topk_select_prev(const spc_dims* d, const float* spec_logits, const float* lse, int32_t k,
                                int32_t* idx, uint32_t* bitmap, const int32_t* prev_idx, int32_t prev_k,
                                int32_t* src, spc_stream stream) {
  const spc_status st = check_topk_args(d, spec_logits, lse, k, idx, bitmap);
  if (st != SPC_OK) return st;
  if (prev_k < 0 || prev_k > (1 << 24)) return SPC_ERR_INVALID;
  if (k > 0 && (src == nullptr ||
                (prev_k > 0 && (prev_idx == nullptr || overlap(prev_idx, (size_t)d->B * d->Hkv * prev_k * 4, idx,
                                                               (size_t)d->B * d->Hkv * k * 4)))))
    return SPC_ERR_INVALID;
  if (d->q_groups_cap == 0 && k == 0) return SPC_OK;
  return spc::launch_topk(d, spec_logits, lse, k, idx, bitmap, reinterpret_cast<cudaStream_t>(stream), prev_idx,
                          prev_k, k > 0 ? src : nullptr);
}

spc_status spc_host_gather(const spc_dims* d, const uint16_t* host_kv, int64_t n_cap, const int32_t* idx,
                           int32_t k, uint16_t* staging, int32_t max_ctas, spc_stream stream) {
  spc_status st = check_dims(d);
  if (st != SPC_OK) return st;
  if (k < 0 || n_cap < 0 || max_ctas < 0) return SPC_ERR_INVALID;
  if (k == 0) return SPC_OK;
  if (host_kv == nullptr || idx == nullptr || staging == nullptr) return SPC_ERR_INVALID;
  if (!aligned16(host_kv) || !aligned16(staging)) return SPC_ERR_INVALID;
  const void* dev = nullptr;
  st = mapped_device_pointer(host_kv, &dev);
  if (st != SPC_OK) return st;
  return spc::launch_host_gather(d, static_cast<const uint16_t*>(dev), n_cap, idx, k, staging, max_ctas,
                                 reinterpret_cast<cudaStream_t>(stream));
}


spc_status spc_host_gather_prev(const spc_dims* d, const uint16_t* host_kv, int64_t n_cap, const int32_t* idx,
                                int32_t k, uint16_t* staging, const int32_t* src, const uint16_t* prev_staging,
                                int32_t prev_k, int32_t max_ctas, spc_stream stream) {
  spc_status st = check_dims(d);
  if (st != SPC_OK) return st;
  if (k < 0 || n_cap < 0 || max_ctas < 0 || prev_k < 0 || prev_k > (1 << 24)) return SPC_ERR_INVALID;
  if (k == 0) return SPC_OK;
  if (host_kv == nullptr || idx == nullptr || staging == nullptr || src == nullptr) return SPC_ERR_INVALID;
  if (!aligned16(host_kv) || !aligned16(staging)) return SPC_ERR_INVALID;
  if (prev_k > 0 && (prev_staging == nullptr || !aligned16(prev_staging) ||
                     overlap(prev_staging, staging_bytes(d, prev_k), staging, staging_bytes(d, k))))
    return SPC_ERR_INVALID;
  const void* dev = nullptr;
  st = mapped_device_pointer(host_kv, &dev);
  if (st != SPC_OK) return st;
  return spc::launch_host_gather(d, static_cast<const uint16_t*>(dev), n_cap, idx, k, staging, max_ctas,
                                 reinterpret_cast<cudaStream_t>(stream), src,
                                 prev_k > 0 ? prev_staging : nullptr, prev_k);
}

}  // extern "C"

// ---------------------------------------------------------------- the prompt path
namespace {

// On the boundary of a 4-byte element, as an int32 or binary32 array has to be.
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A view of [b][t][h][128] whose rows lie on 16-byte boundaries and apart from
// one another: each stride, smallest first, clears what the smaller ones span
// (an axis of one element is never stepped along).
bool layout_ok(const spc_layout& l, int64_t nb, int64_t nt, int64_t nh) {
  const int64_t lim = (int64_t)1 << 38;  // elements: 2^39 bytes, within a TMA stride's range
  if (l.b % 8 != 0 || l.t % 8 != 0 || l.h % 8 != 0) return false;
  if (l.b < 0 || l.t < 0 || l.h < 0 || l.b >= lim || l.t >= lim || l.h >= lim) return false;
  int64_t st[3] = {l.b, l.t, l.h}, n[3] = {nb, nt, nh};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (st[j] > st[j + 1]) {
        std::swap(st[j], st[j + 1]);
        std::swap(n[j], n[j + 1]);
      }
  int64_t span = spc::kD;
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (st[i] < span) return false;
    span += st[i] * (n[i] - 1);  // below 2^38 * 2^31
    if (span >= ((int64_t)1 << 60)) return false;
  }
  return true;
}

// Bytes from the view's first element to behind its last.
size_t layout_bytes(const spc_layout& l, int64_t nb, int64_t nt, int64_t nh) {
  if (nb <= 0 || nt <= 0 || nh <= 0) return 0;
  return 2 * (size_t)((nb - 1) * l.b + (nt - 1) * l.t + (nh - 1) * l.h + spc::kD);
}

// Whether a row of one view of [nb][nt][heads][128] shares a byte with a row of
// the other.  Told exactly where an axis that both step along has one stride
// (views of one buffer; heads may differ): the distance of two rows is then the
// views' distance less some steps along the axes, and as each stride clears
// what the smaller ones span, only the two whole numbers of steps next to the
// distance that is left can come within a row of it, largest stride first.
// Views of other strides that reach into one another: by their first rows.
bool rows_meet(const uint16_t* a, const spc_layout& la, int64_t ha, const uint16_t* b, const spc_layout& lb, int64_t hb,
               int64_t nb, int64_t nt) {
  if (!overlap(a, layout_bytes(la, nb, nt, ha), b, layout_bytes(lb, nb, nt, hb))) return false;
  const spc_layout l = {la.b, la.t, ha > 1 ? la.h : lb.h};
  if ((nb > 1 && la.b != lb.b) || (nt > 1 && la.t != lb.t) || (ha > 1 && hb > 1 && la.h != lb.h) ||
      !layout_ok(l, nb, nt, std::max(ha, hb)))
    return overlap(a, 2 * spc::kD, b, 2 * spc::kD);
  struct Axis {
    int64_t step, least, most;  // bytes; the difference of two rows' indices
  } ax[3] = {{2 * l.b, 1 - nb, nb - 1}, {2 * l.t, 1 - nt, nt - 1}, {2 * l.h, 1 - hb, ha - 1}};
  for (Axis& x : ax)
    if (x.least == 0 && x.most == 0) x.step = 0;
  std::sort(ax, ax + 3, [](const Axis& x, const Axis& y) { return x.step > y.step; });
  const int64_t apart = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  for (int pick = 0; pick < 8; ++pick) {
    int64_t left = apart;
    bool inside = true;
    for (int i = 0; i < 3 && ax[i].step > 0; ++i) {
      int64_t n = left / ax[i].step - (left % ax[i].step < 0) + ((pick >> i) & 1);
      inside = inside && n >= ax[i].least && n <= ax[i].most;
      left -= n * ax[i].step;
    }
    if (inside && left < 2 * spc::kD && left > -2 * spc::kD) return true;
  }
  return false;
}

bool same_layout(const spc_layout& x, const spc_layout& y) { return x.b == y.b && x.t == y.t && x.h == y.h; }

}  // namespace

extern "C" {

spc_status spc_rope_frequencies(const spc_rope_scaling* s, int32_t rot, uint64_t* turns, float* mscale) {
  if (s == nullptr || turns == nullptr || mscale == nullptr) return SPC_ERR_INVALID;
  if (rot < 16 || rot > spc::kD || rot % 16 != 0) return SPC_ERR_UNSUPPORTED;
  if (s->kind < SPC_ROPE_PLAIN || s->kind > SPC_ROPE_RAMP) return SPC_ERR_INVALID;
  if (!(std::isfinite(s->theta) && s->theta > 1.0)) return SPC_ERR_INVALID;
  if (s->kind != SPC_ROPE_PLAIN && !(std::isfinite(s->factor) && s->factor >= 1.0)) return SPC_ERR_INVALID;
  const bool by_turns = s->kind == SPC_ROPE_BANDS || s->kind == SPC_ROPE_RAMP;
  if (by_turns && !(std::isfinite(s->high) && std::isfinite(s->context) && s->low > 0.0 && s->low < s->high &&
                    s->context > 0.0))
    return SPC_ERR_INVALID;
  const double two_pi = 6.283185307179586476925286766559;
  double from = 0.0, to = 0.0;  // RAMP: the pairs between which it falls
  if (s->kind == SPC_ROPE_RAMP) {
    const auto pair_of = [&](double n) { return rot * std::log(s->context / (n * two_pi)) / (2.0 * std::log(s->theta)); };
    from = std::max(std::floor(pair_of(s->high)), 0.0);
    to = std::min(std::ceil(pair_of(s->low)), (double)(rot - 1));
  }
  for (int32_t i = 0; i < rot / 2; ++i) {
    double f = std::pow(s->theta, -2.0 * i / rot);
    if (s->kind == SPC_ROPE_LINEAR) {
      f /= s->factor;
    } else if (s->kind == SPC_ROPE_BANDS) {
      const double n = s->context * f / two_pi;
      const double mix = std::min(1.0, std::max(0.0, (n - s->low) / (s->high - s->low)));
      f = (1.0 - mix) * f / s->factor + mix * f;
    } else if (s->kind == SPC_ROPE_RAMP) {
      const double ramp = std::min(1.0, std::max(0.0, (i - from) / std::max(to - from, 0.001)));
      f = f / s->factor * ramp + f * (1.0 - ramp);
    }
    turns[i] = (uint64_t)(f / two_pi * 18446744073709551616.0);  // f <= 1: below 2^62
  }
  *mscale = s->kind == SPC_ROPE_RAMP ? (float)(0.1 * std::log(s->factor) + 1.0) : 1.0f;
  return SPC_OK;
}

// The checks of a call's arguments come back with `nothing` set where there is
// nothing to do.
static spc_status check_rope(const spc_rope_dims* d, const int32_t* pos, const uint64_t* turns, const uint16_t* q,
                             const uint16_t* k, const uint16_t* v, const uint16_t* q_out, const uint16_t* k_out,
                             const uint16_t* v_out, bool& nothing) {
  nothing = false;
  if (d == nullptr || d->B <= 0 || d->T < 0 || d->Hq < 0 || d->Hkv < 0 || d->D <= 0) return SPC_ERR_INVALID;
  if (d->Hq > (1 << 16) || d->Hkv > (1 << 16)) return SPC_ERR_INVALID;
  if (d->interleaved != 0 && d->interleaved != 1) return SPC_ERR_INVALID;
  if (!std::isfinite(d->mscale)) return SPC_ERR_INVALID;
  if (d->D != spc::kD || d->rot < 16 || d->rot > spc::kD || d->rot % 16 != 0) return SPC_ERR_UNSUPPORTED;
  if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr) ||
      (v == nullptr) != (v_out == nullptr))
    return SPC_ERR_INVALID;
  if (d->T == 0) {
    nothing = true;
    return SPC_OK;
  }
  if ((q == nullptr) != (d->Hq == 0) || (k == nullptr) != (d->Hkv == 0) || (v != nullptr && d->Hkv == 0))
    return SPC_ERR_INVALID;
  if (q == nullptr && k == nullptr) {
    nothing = true;
    return SPC_OK;
  }
  if (pos == nullptr || turns == nullptr || !aligned4(pos) || (reinterpret_cast<uintptr_t>(turns) & 7u) != 0)
    return SPC_ERR_INVALID;
  const struct {
    const uint16_t *in, *out;
    const spc_layout *li, *lo;
    int32_t heads;
  } rows[3] = {{q, q_out, &d->q, &d->q_out, d->Hq},
               {k, k_out, &d->k, &d->k_out, d->Hkv},
               {v, v_out, &d->v, &d->v_out, d->Hkv}};
  for (const auto& r : rows) {
    if (r.in == nullptr) continue;
    if (!aligned16(r.in) || !aligned16(r.out)) return SPC_ERR_INVALID;
    if (!layout_ok(*r.li, d->B, d->T, r.heads) || !layout_ok(*r.lo, d->B, d->T, r.heads)) return SPC_ERR_INVALID;
    // in place is the same view; any other output that reaches into its input would race with the reads
    if (!(r.in == r.out && same_layout(*r.li, *r.lo)) &&
        overlap(r.in, layout_bytes(*r.li, d->B, d->T, r.heads), r.out, layout_bytes(*r.lo, d->B, d->T, r.heads)))
      return SPC_ERR_INVALID;
  }
  for (const auto& r : rows)  // nor may an output's rows lie on another tensor's
    for (const auto& x : rows)
      if (&r != &x && (rows_meet(r.out, *r.lo, r.heads, x.in, *x.li, x.heads, d->B, d->T) ||
                       rows_meet(r.out, *r.lo, r.heads, x.out, *x.lo, x.heads, d->B, d->T)))
        return SPC_ERR_INVALID;
  return SPC_OK;
}

spc_status spc_rope_check(const spc_rope_dims* d, const int32_t* pos, const uint64_t* turns, const uint16_t* q,
                          const uint16_t* k, const uint16_t* v, uint16_t* q_out, uint16_t* k_out, uint16_t* v_out,
                          spc_stream) {
  bool nothing;
  return check_rope(d, pos, turns, q, k, v, q_out, k_out, v_out, nothing);
}

spc_status spc_rope(const spc_rope_dims* d, const int32_t* pos, const uint64_t* turns, const uint16_t* q,
                    const uint16_t* k, const uint16_t* v, uint16_t* q_out, uint16_t* k_out, uint16_t* v_out,
                    spc_stream stream) {
  bool nothing;
  const spc_status st = check_rope(d, pos, turns, q, k, v, q_out, k_out, v_out, nothing);
  if (st != SPC_OK || nothing) return st;
  return spc::launch_rope(d, pos, turns, q, k, v, q_out, k_out, v_out, reinterpret_cast<cudaStream_t>(stream));
}

spc_status spc_rope_axes(const int32_t* sections, int32_t axes, int32_t order, int32_t rot, uint8_t* axis) {
  if (sections == nullptr || axis == nullptr || axes < 1 || axes > 4) return SPC_ERR_INVALID;
  if (order != SPC_AXIS_SECTIONS && order != SPC_AXIS_TURNS) return SPC_ERR_INVALID;
  if (rot < 16 || rot > spc::kD || rot % 16 != 0) return SPC_ERR_UNSUPPORTED;
  int64_t sum = 0;
  for (int32_t a = 0; a < axes; ++a) {
    if (sections[a] < 0) return SPC_ERR_INVALID;
    sum += sections[a];
  }
  if (sum != rot / 2) return SPC_ERR_INVALID;
  uint8_t of[spc::kD / 2];
  int32_t count[4] = {0, 0, 0, 0}, section = 0, left = sections[0];
  for (int32_t i = 0; i < rot / 2; ++i) {
    if (order == SPC_AXIS_SECTIONS) {
      while (left == 0) left = sections[++section];
      --left;
      of[i] = (uint8_t)section;
    } else {
      of[i] = (uint8_t)(i < axes * sections[i % axes] ? i % axes : 0);
    }
    ++count[of[i]];
  }
  for (int32_t a = 0; a < axes; ++a)
    if (count[a] != sections[a]) return SPC_ERR_INVALID;
  std::copy(of, of + rot / 2, axis);
  return SPC_OK;
}

static spc_status check_norm_rope(const spc_norm_rope_dims* d, const int32_t* pos, const uint64_t* turns,
                                  const float* q_weight, const float* k_weight, const uint16_t* q, const uint16_t* k,
                                  const uint16_t* v, const uint16_t* q_out, const uint16_t* k_out,
                                  const uint16_t* v_out, bool& nothing) {
  nothing = false;
  if (d == nullptr) return SPC_ERR_INVALID;
  const spc_status st = check_rope(&d->rope, pos, turns, q, k, v, q_out, k_out, v_out, nothing);
  if (st != SPC_OK) return st;
  if (d->axes < 1 || d->axes > 4) return SPC_ERR_INVALID;
  for (int32_t i = 0; i < d->rope.rot / 2; ++i)
    if (d->axis[i] >= d->axes) return SPC_ERR_INVALID;
  if ((q_weight != nullptr || k_weight != nullptr) && !(std::isfinite(d->eps) && d->eps >= 1e-30f))
    return SPC_ERR_INVALID;
  if (nothing) return SPC_OK;
  if ((q_weight != nullptr && q == nullptr) || (k_weight != nullptr && k == nullptr)) return SPC_ERR_INVALID;
  if (!aligned4(q_weight) || !aligned4(k_weight)) return SPC_ERR_INVALID;
  return SPC_OK;
}

spc_status spc_norm_rope_check(const spc_norm_rope_dims* d, const int32_t* pos, const uint64_t* turns,
                               const float* q_weight, const float* k_weight, const uint16_t* q, const uint16_t* k,
                               const uint16_t* v, uint16_t* q_out, uint16_t* k_out, uint16_t* v_out, spc_stream) {
  bool nothing;
  return check_norm_rope(d, pos, turns, q_weight, k_weight, q, k, v, q_out, k_out, v_out, nothing);
}

spc_status spc_norm_rope(const spc_norm_rope_dims* d, const int32_t* pos, const uint64_t* turns, const float* q_weight,
                         const float* k_weight, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                         uint16_t* q_out, uint16_t* k_out, uint16_t* v_out, spc_stream stream) {
  bool nothing;
  const spc_status st =
      check_norm_rope(d, pos, turns, q_weight, k_weight, q, k, v, q_out, k_out, v_out, nothing);
  if (st != SPC_OK || nothing) return st;
  return spc::launch_norm_rope(d, pos, turns, q_weight, k_weight, q, k, v, q_out, k_out, v_out,
                               reinterpret_cast<cudaStream_t>(stream));
}

static spc_status check_prompt_dims(const spc_prompt_dims* d) {
  if (d == nullptr || d->S <= 0 || d->Hq <= 0 || d->Hkv <= 0 || d->D <= 0 || d->q_tokens < 0 || d->k_tokens < 0 ||
      d->q_max < 0 || d->k_max < 0 || d->q_max > d->q_tokens || d->k_max > d->k_tokens)
    return SPC_ERR_INVALID;
  if (d->Hq % d->Hkv != 0 || !(std::isfinite(d->scale) && d->scale > 0.f)) return SPC_ERR_INVALID;
  if (d->D != spc::kD || d->Hq / d->Hkv > 128) return SPC_ERR_UNSUPPORTED;
  if (d->q_tokens >= (1 << 30) || d->k_tokens >= (1 << 30)) return SPC_ERR_UNSUPPORTED;
  if (d->S > 1 && ((d->q.b == 0) != (d->o.b == 0) || (d->k.b == 0) != (d->v.b == 0))) return SPC_ERR_INVALID;
  const int64_t qb = d->q.b ? d->S : 1, kb = d->k.b ? d->S : 1;
  if (!layout_ok(d->q, qb, d->q_tokens, d->Hq) || !layout_ok(d->o, qb, d->q_tokens, d->Hq) ||
      !layout_ok(d->k, kb, d->k_tokens, d->Hkv) || !layout_ok(d->v, kb, d->k_tokens, d->Hkv))
    return SPC_ERR_INVALID;
  // the grid numbers pairs of query tiles, KV heads, sequences and splits
  const int64_t pairs = (int64_t)d->q_max * (d->Hq / d->Hkv) / 128 + 2;
  if ((int64_t)d->S * d->Hkv > (1 << 30) / pairs) return SPC_ERR_UNSUPPORTED;
  return SPC_OK;
}

size_t spc_prompt_attn_workspace_bytes(const spc_prompt_dims* d) {
  return check_prompt_dims(d) == SPC_OK ? spc::prompt_workspace_bytes(d) : 0;
}

// A range of bytes that a call reads.
struct Bytes {
  const void* p;
  size_t n;
};

// need: workspace of the call (a valid shape's); more: what it reads besides.
static spc_status check_attn(const spc_prompt_dims* d, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                             const int32_t* q_begin, const int32_t* q_len, const int32_t* k_begin,
                             const int32_t* k_len, const uint16_t* o, const float* lse, const void* ws,
                             size_t ws_bytes, size_t need, const Bytes (&more)[2], bool& nothing) {
  nothing = false;
  if (d->q_max == 0) {
    nothing = true;
    return SPC_OK;
  }
  if (d->S > 1 && d->q.b == 0 && q_begin == nullptr) return SPC_ERR_INVALID;  // all on the same query rows
  if (q == nullptr || o == nullptr || (d->k_max > 0 && (k == nullptr || v == nullptr))) return SPC_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return SPC_ERR_INVALID;
  if (!aligned4(q_begin) || !aligned4(q_len) || !aligned4(k_begin) || !aligned4(k_len) || !aligned4(lse))
    return SPC_ERR_INVALID;
  if ((ws == nullptr && (need > 256 || ws_bytes != 0)) || !aligned16(ws)) return SPC_ERR_INVALID;
  if (ws != nullptr && ws_bytes < need) return SPC_ERR_WORKSPACE;
  const int64_t qb = d->q.b ? d->S : 1, kb = d->k.b ? d->S : 1;
  // what the call writes shares no byte range with what it reads or writes besides
  const Bytes part[8] = {{q, layout_bytes(d->q, qb, d->q_tokens, d->Hq)},
                         {k, layout_bytes(d->k, kb, d->k_tokens, d->Hkv)},
                         {v, layout_bytes(d->v, kb, d->k_tokens, d->Hkv)},
                         more[0],
                         more[1],
                         {o, layout_bytes(d->o, qb, d->q_tokens, d->Hq)},
                         {lse, (size_t)qb * d->q_tokens * d->Hq * sizeof(float)},
                         {ws, need}};
  for (int i = 5; i < 8; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(part[i].p, part[i].n, part[j].p, part[j].n)) return SPC_ERR_INVALID;
  return SPC_OK;
}

static spc_status check_prompt_attn(const spc_prompt_dims* d, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                    const int32_t* q_begin, const int32_t* q_len, const int32_t* k_begin,
                                    const int32_t* k_len, const uint16_t* o, const float* lse, const void* ws,
                                    size_t ws_bytes, bool& nothing) {
  nothing = false;
  const spc_status st = check_prompt_dims(d);
  if (st != SPC_OK) return st;
  return check_attn(d, q, k, v, q_begin, q_len, k_begin, k_len, o, lse, ws, ws_bytes, spc::prompt_workspace_bytes(d),
                    {{nullptr, 0}, {nullptr, 0}}, nothing);
}

spc_status spc_prompt_attn_check(const spc_prompt_dims* d, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                 const int32_t* q_begin, const int32_t* q_len, const int32_t* k_begin,
                                 const int32_t* k_len, uint16_t* o, float* lse, void* ws, size_t ws_bytes, spc_stream) {
  bool nothing;
  return check_prompt_attn(d, q, k, v, q_begin, q_len, k_begin, k_len, o, lse, ws, ws_bytes, nothing);
}

spc_status spc_prompt_attn(const spc_prompt_dims* d, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                           const int32_t* q_begin, const int32_t* q_len, const int32_t* k_begin,
                           const int32_t* k_len, uint16_t* o, float* lse, void* ws, size_t ws_bytes,
                           spc_stream stream) {
  bool nothing;
  const spc_status st = check_prompt_attn(d, q, k, v, q_begin, q_len, k_begin, k_len, o, lse, ws, ws_bytes, nothing);
  if (st != SPC_OK || nothing) return st;
  return spc::launch_prompt_attn(d, q, k, v, q_begin, q_len, k_begin, k_len, o, lse, ws,
                                 reinterpret_cast<cudaStream_t>(stream));
}

// Page-locked words for one call's copies from the device, so that several are in flight before one wait (three copies to
// pageable memory, each of which waits, took 33 us, one 15; three of these 16).  Kept for later calls.
class StatusWords {
 public:
  StatusWords() {
    const std::lock_guard<std::mutex> lock(mu_);
    if (kept_ > 0) p_ = idle_[--kept_];
  }
  ~StatusWords() {
    if (p_ == nullptr) return;
    const std::lock_guard<std::mutex> lock(mu_);
    if (kept_ < kMost)
      idle_[kept_++] = p_;
    else
      cudaFreeHost(p_);
  }
  StatusWords(const StatusWords&) = delete;
  StatusWords& operator=(const StatusWords&) = delete;
  cudaError_t get(volatile uint32_t** p) {
    cudaError_t e = cudaSuccess;
    if (p_ == nullptr) {
      cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;  // another thread's capture may go on
      cudaThreadExchangeStreamCaptureMode(&mode);
      void* words = nullptr;
      e = cudaHostAlloc(&words, 4 * sizeof(uint32_t), cudaHostAllocPortable);
      cudaThreadExchangeStreamCaptureMode(&mode);
      if (e == cudaSuccess) p_ = static_cast<uint32_t*>(words);
    }
    *p = p_;
    return e;
  }

 private:
  static constexpr int kMost = 16;
  static inline std::mutex mu_;
  static inline uint32_t* idle_[kMost] = {};
  static inline int kept_ = 0;
  uint32_t* p_ = nullptr;
};

spc_status spc_prompt_attn_status(void* ws, spc_stream stream) {
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void* word[3] = {ws, nullptr, nullptr};
  StatusWords words;
  volatile uint32_t* v = nullptr;
  cudaError_t e = words.get(&v);
  if (ws == nullptr) {  // the device's words, one of each kind of call
    if (e == cudaSuccess) e = spc::prompt_fault_word(&word[0]);
    if (e == cudaSuccess) e = spc::window_fault_word(&word[1]);
    if (e == cudaSuccess) e = spc::prefix_fault_word(&word[2]);
  }
  const int n = ws == nullptr ? 3 : 1;
  for (int i = 0; i < n && e == cudaSuccess; ++i)
    e = cudaMemcpyAsync(const_cast<uint32_t*>(v + i), word[i], sizeof(uint32_t), cudaMemcpyDeviceToHost, s);
  const cudaError_t ended = v != nullptr ? cudaStreamSynchronize(s) : e;  // also behind a copy that was refused
  if (e == cudaSuccess) e = ended;
  bool found = false;
  for (int i = 0; i < n && e == cudaSuccess; ++i)
    if (v[i] != 0u) {
      found = true;
      e = cudaMemsetAsync(word[i], 0, sizeof(uint32_t), s);
    }
  if (e == cudaSuccess && found) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) {
    spc_host::set_cuda_error(e);
    return SPC_ERR_CUDA;
  }
  return found ? SPC_ERR_TIMEOUT : SPC_OK;
}

int64_t spc_prompt_attn_wait_limit(int64_t ns) { return spc::prompt_wait_limit(ns); }

static spc_status check_window(const spc_prompt_dims* d, int32_t window, int32_t sinks) {
  const spc_status st = check_prompt_dims(d);
  if (st != SPC_OK) return st;
  return window < 1 || sinks < 0 ? SPC_ERR_INVALID : SPC_OK;
}

size_t spc_window_attn_workspace_bytes(const spc_prompt_dims* d, int32_t window, int32_t sinks) {
  if (check_window(d, window, sinks) != SPC_OK) return 0;
  return window >= d->k_max ? spc::prompt_workspace_bytes(d) : spc::window_workspace_bytes(d, window, sinks);
}

static spc_status check_window_attn(const spc_prompt_dims* d, int32_t window, int32_t sinks, const uint16_t* q,
                                    const uint16_t* k, const uint16_t* v, const int32_t* q_begin,
                                    const int32_t* q_len, const int32_t* k_begin, const int32_t* k_len,
                                    const uint16_t* o, const float* lse, const void* ws, size_t ws_bytes,
                                    bool& nothing) {
  nothing = false;
  const spc_status st = check_window(d, window, sinks);
  if (st != SPC_OK) return st;
  return check_attn(d, q, k, v, q_begin, q_len, k_begin, k_len, o, lse, ws, ws_bytes,
                    spc_window_attn_workspace_bytes(d, window, sinks), {{nullptr, 0}, {nullptr, 0}}, nothing);
}

spc_status spc_window_attn_check(const spc_prompt_dims* d, int32_t window, int32_t sinks, const uint16_t* q,
                                 const uint16_t* k, const uint16_t* v, const int32_t* q_begin, const int32_t* q_len,
                                 const int32_t* k_begin, const int32_t* k_len, uint16_t* o, float* lse, void* ws,
                                 size_t ws_bytes, spc_stream) {
  bool nothing;
  return check_window_attn(d, window, sinks, q, k, v, q_begin, q_len, k_begin, k_len, o, lse, ws, ws_bytes, nothing);
}

spc_status spc_window_attn(const spc_prompt_dims* d, int32_t window, int32_t sinks, const uint16_t* q,
                           const uint16_t* k, const uint16_t* v, const int32_t* q_begin, const int32_t* q_len,
                           const int32_t* k_begin, const int32_t* k_len, uint16_t* o, float* lse, void* ws,
                           size_t ws_bytes, spc_stream stream) {
  bool nothing;
  const spc_status st =
      check_window_attn(d, window, sinks, q, k, v, q_begin, q_len, k_begin, k_len, o, lse, ws, ws_bytes, nothing);
  if (st != SPC_OK || nothing) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (window >= d->k_max) return spc::launch_prompt_attn(d, q, k, v, q_begin, q_len, k_begin, k_len, o, lse, ws, s);
  return spc::launch_window_attn(d, window, sinks, q, k, v, q_begin, q_len, k_begin, k_len, o, lse, ws, s);
}

static spc_status check_prefix(const spc_prompt_dims* d, const spc_prefix* p) {
  const spc_status st = check_prompt_dims(d);
  if (st != SPC_OK) return st;
  if (p == nullptr || p->tokens < 0) return SPC_ERR_INVALID;
  if (p->tokens >= (1 << 30)) return SPC_ERR_UNSUPPORTED;
  if (!layout_ok(p->k, 1, p->tokens, d->Hkv) || !layout_ok(p->v, 1, p->tokens, d->Hkv)) return SPC_ERR_INVALID;
  return SPC_OK;
}

size_t spc_prefix_attn_workspace_bytes(const spc_prompt_dims* d, const spc_prefix* p) {
  if (check_prefix(d, p) != SPC_OK) return 0;
  return p->tokens == 0 ? spc::prompt_workspace_bytes(d) : spc::prefix_workspace_bytes(d, p);
}

int32_t spc_prefix_attn_together(const spc_prompt_dims* d, const spc_prefix* p, int32_t placed) {
  return check_prefix(d, p) != SPC_OK ? 0 : spc::prefix_together(d, p, placed != 0);
}

static spc_status check_prefix_attn(const spc_prompt_dims* d, const spc_prefix* p, const uint16_t* q,
                                    const uint16_t* pk, const uint16_t* pv, const int32_t* p_len, const uint16_t* k,
                                    const uint16_t* v, const int32_t* q_begin, const int32_t* q_len,
                                    const int32_t* k_begin, const int32_t* k_len, const uint16_t* o, const float* lse,
                                    const void* ws, size_t ws_bytes, bool& nothing) {
  nothing = false;
  spc_status st = check_prefix(d, p);
  if (st != SPC_OK) return st;
  st = check_attn(d, q, k, v, q_begin, q_len, k_begin, k_len, o, lse, ws, ws_bytes, spc_prefix_attn_workspace_bytes(d, p),
                  {{pk, layout_bytes(p->k, 1, p->tokens, d->Hkv)}, {pv, layout_bytes(p->v, 1, p->tokens, d->Hkv)}},
                  nothing);
  if (st != SPC_OK || nothing) return st;
  if (p->tokens > 0 && (pk == nullptr || pv == nullptr)) return SPC_ERR_INVALID;
  return !aligned16(pk) || !aligned16(pv) || !aligned4(p_len) ? SPC_ERR_INVALID : SPC_OK;
}

spc_status spc_prefix_attn_check(const spc_prompt_dims* d, const spc_prefix* p, const uint16_t* q, const uint16_t* pk,
                                 const uint16_t* pv, const int32_t* p_len, const uint16_t* k, const uint16_t* v,
                                 const int32_t* q_begin, const int32_t* q_len, const int32_t* k_begin,
                                 const int32_t* k_len, uint16_t* o, float* lse, void* ws, size_t ws_bytes, spc_stream) {
  bool nothing;
  return check_prefix_attn(d, p, q, pk, pv, p_len, k, v, q_begin, q_len, k_begin, k_len, o, lse, ws, ws_bytes, nothing);
}

spc_status spc_prefix_attn(const spc_prompt_dims* d, const spc_prefix* p, const uint16_t* q, const uint16_t* pk,
                           const uint16_t* pv, const int32_t* p_len, const uint16_t* k, const uint16_t* v,
                           const int32_t* q_begin, const int32_t* q_len, const int32_t* k_begin,
                           const int32_t* k_len, uint16_t* o, float* lse, void* ws, size_t ws_bytes,
                           spc_stream stream) {
  bool nothing;
  const spc_status st =
      check_prefix_attn(d, p, q, pk, pv, p_len, k, v, q_begin, q_len, k_begin, k_len, o, lse, ws, ws_bytes, nothing);
  if (st != SPC_OK || nothing) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p->tokens == 0) return spc::launch_prompt_attn(d, q, k, v, q_begin, q_len, k_begin, k_len, o, lse, ws, s);
  return spc::launch_prefix_attn(d, p, q, pk, pv, p_len, k, v, q_begin, q_len, k_begin, k_len, o, lse, ws, s);
}

// host_dev: the device's address of host_kv.
static spc_status check_extend(const spc_dims* d, int32_t n, const uint16_t* k_new, const uint16_t* v_new,
                               const spc_layout* k_layout, const spc_layout* v_layout, const void* records,
                               const uint16_t* resid, const uint16_t* host_kv, int64_t n_cap, const void** host_dev) {
  spc_status st = check_dims(d);
  if (st != SPC_OK) return st;
  if (n < 0 || (int64_t)d->N + n > (1 << 30)) return SPC_ERR_INVALID;
  if (n == 0) return SPC_OK;
  spc_dims after = *d;
  after.N += n;
  st = check_dims(&after);  // the capacities hold the extended cache
  if (st != SPC_OK) return st;
  const int32_t nq = spc::num_quantized(d->N, d->R, d->group), nq1 = spc::num_quantized(after.N, d->R, d->group);
  if (k_new == nullptr || v_new == nullptr || k_layout == nullptr || v_layout == nullptr) return SPC_ERR_INVALID;
  if (nq1 > nq && records == nullptr) return SPC_ERR_INVALID;
  if ((d->N > nq || after.N > nq1) && resid == nullptr) return SPC_ERR_INVALID;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(records) || !aligned16(resid) || !aligned16(host_kv))
    return SPC_ERR_INVALID;
  if (!layout_ok(*k_layout, d->B, n, d->Hkv) || !layout_ok(*v_layout, d->B, n, d->Hkv)) return SPC_ERR_INVALID;
  const size_t res = spc_resid_bytes(d), rec = spc_records_bytes(d);
  const size_t kb = layout_bytes(*k_layout, d->B, n, d->Hkv), vb = layout_bytes(*v_layout, d->B, n, d->Hkv);
  if (overlap(k_new, kb, resid, res) || overlap(v_new, vb, resid, res) || overlap(k_new, kb, records, rec) ||
      overlap(v_new, vb, records, rec))
    return SPC_ERR_INVALID;
  if (host_kv != nullptr) {
    if (n_cap < after.N) return SPC_ERR_INVALID;
    return mapped_device_pointer(host_kv, host_dev);
  }
  return SPC_OK;
}

spc_status spc_extend_kv_check(const spc_dims* d, int32_t n, const uint16_t* k_new, const uint16_t* v_new,
                               const spc_layout* k_layout, const spc_layout* v_layout, void* records, uint16_t* resid,
                               uint16_t* host_kv, int64_t n_cap, spc_stream) {
  const void* host_dev = nullptr;
  return check_extend(d, n, k_new, v_new, k_layout, v_layout, records, resid, host_kv, n_cap, &host_dev);
}

spc_status spc_extend_kv(const spc_dims* d, int32_t n, const uint16_t* k_new, const uint16_t* v_new,
                         const spc_layout* k_layout, const spc_layout* v_layout, void* records, uint16_t* resid,
                         uint16_t* host_kv, int64_t n_cap, spc_stream stream) {
  const void* host_dev = nullptr;
  const spc_status st =
      check_extend(d, n, k_new, v_new, k_layout, v_layout, records, resid, host_kv, n_cap, &host_dev);
  if (st != SPC_OK || n == 0) return st;
  return spc::launch_extend(d, n, k_new, v_new, k_layout, v_layout, records, resid,
                            static_cast<uint16_t*>(const_cast<void*>(host_dev)), n_cap,
                            reinterpret_cast<cudaStream_t>(stream));
}

static spc_status check_dequantize(const spc_dims* d, const void* records, const uint16_t* resid, int32_t first,
                                   int32_t n, const uint16_t* k, const uint16_t* v, const spc_layout* k_layout,
                                   const spc_layout* v_layout) {
  const spc_status st = check_dims(d);
  if (st != SPC_OK) return st;
  if (first < 0 || n < 0 || (int64_t)first + n > d->N) return SPC_ERR_INVALID;
  if (n == 0) return SPC_OK;
  const int32_t nq = spc::num_quantized(d->N, d->R, d->group);
  if (k == nullptr || v == nullptr || k_layout == nullptr || v_layout == nullptr) return SPC_ERR_INVALID;
  if ((first < nq && records == nullptr) || (first + n > nq && resid == nullptr)) return SPC_ERR_INVALID;
  if (!aligned16(k) || !aligned16(v) || !aligned16(records) || !aligned16(resid)) return SPC_ERR_INVALID;
  if (!layout_ok(*k_layout, d->B, n, d->Hkv) || !layout_ok(*v_layout, d->B, n, d->Hkv)) return SPC_ERR_INVALID;
  const size_t res = spc_resid_bytes(d), rec = spc_records_bytes(d);
  const size_t kb = layout_bytes(*k_layout, d->B, n, d->Hkv), vb = layout_bytes(*v_layout, d->B, n, d->Hkv);
  if (overlap(k, kb, resid, res) || overlap(v, vb, resid, res) || overlap(k, kb, records, rec) ||
      overlap(v, vb, records, rec) ||
      rows_meet(k, *k_layout, d->Hkv, v, *v_layout, d->Hkv, d->B, n))
    return SPC_ERR_INVALID;
  return SPC_OK;
}

spc_status spc_dequantize_kv_check(const spc_dims* d, const void* records, const uint16_t* resid, int32_t first,
                                   int32_t n, uint16_t* k, uint16_t* v, const spc_layout* k_layout,
                                   const spc_layout* v_layout, spc_stream) {
  return check_dequantize(d, records, resid, first, n, k, v, k_layout, v_layout);
}

spc_status spc_dequantize_kv(const spc_dims* d, const void* records, const uint16_t* resid, int32_t first, int32_t n,
                             uint16_t* k, uint16_t* v, const spc_layout* k_layout, const spc_layout* v_layout,
                             spc_stream stream) {
  const spc_status st = check_dequantize(d, records, resid, first, n, k, v, k_layout, v_layout);
  if (st != SPC_OK || n == 0) return st;
  return spc::launch_dequantize(d, records, resid, first, n, k, v, k_layout, v_layout,
                                reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
