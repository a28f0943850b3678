// The causal attention of prompts: see prompt_attn.cuh.
#include <atomic>

#include "prompt_attn.cuh"

namespace spc {
namespace {

std::atomic<int64_t> prompt_limit{2000000000};  // of a wait in the kernels launched from now on, in ns

}  // namespace

// (held to 1000 s, so that no sum of times overflows: mbar_wait)
int64_t prompt_wait_limit(int64_t ns) {
  return ns > 0 ? prompt_limit.exchange(std::min<int64_t>(ns, 1000000000000)) : prompt_limit.load();
}

cudaError_t prompt_fault_word(void** word) { return cudaGetSymbolAddress(word, prompt_device_fault); }

size_t prompt_workspace_bytes(const spc_prompt_dims* d) { return prompt_bytes(d, PromptRule()); }

spc_status launch_prompt_attn(const spc_prompt_dims* d, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                              const int32_t* q_begin, const int32_t* q_len, const int32_t* k_begin,
                              const int32_t* k_len, uint16_t* o, float* lse, void* ws, cudaStream_t stream) {
  return launch_prompt<kPlain>(d, PromptRule(), {q, k, v, q_begin, q_len, k_begin, k_len, o, lse, ws}, stream);
}

}  // namespace spc
