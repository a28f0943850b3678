// The causal attention of prompts with a sliding window and a few first tokens
// that stay visible: a query at place p of its sequence sees the keys j <= p
// with j > p - window or j < sinks.  The kernel of prompt_attn.cuh, walking over
// the first tokens' blocks and then, from the first row's window on, over the
// windows of an item's rows: what lies between is not read.  Single tokens take
// few_attn.cuh's.
#include "few_attn.cuh"

namespace spc {

cudaError_t window_fault_word(void** word) { return cudaGetSymbolAddress(word, prompt_device_fault); }

size_t window_workspace_bytes(const spc_prompt_dims* d, int32_t window, int32_t sinks) {
  if (few_rows(d)) return kPromptHead;
  PromptRule rule;
  rule.window = window;
  rule.sinks = sinks;
  return prompt_bytes(d, rule);
}

spc_status launch_window_attn(const spc_prompt_dims* d, int32_t window, int32_t sinks, const uint16_t* q,
                              const uint16_t* k, const uint16_t* v, const int32_t* q_begin, const int32_t* q_len,
                              const int32_t* k_begin, const int32_t* k_len, uint16_t* o, float* lse, void* ws,
                              cudaStream_t stream) {
  PromptRule rule;
  rule.window = window;
  rule.sinks = sinks;
  const PromptTensors x = {q, k, v, q_begin, q_len, k_begin, k_len, o, lse, ws};
  if (few_rows(d)) {
    PromptArgs a = prompt_args(d, rule, x);
    return launch_few<false>(a, d, stream);
  }
  return launch_prompt<kWindow>(d, rule, x, stream);
}

}  // namespace spc
