// The causal attention of prompts with a sliding window and a few first tokens
// that stay visible: a query at place p of its sequence sees the keys j <= p
// with j > p - window or j < sinks.  The kernel of prompt_attn.cuh, walking over
// the first tokens' blocks and then, from the first row's window on, over the
// windows of an item's rows: what lies between is not read.  Single tokens take
// few_attn.cuh's.
// Long windows are bound by the tensor cores: a 32768-token prompt of 32 and 8
// heads, window 4096, takes 1.46 to 1.50 ms (2.06 TFLOP: 74% of the measured
// burst rate; 0.73 us per 64 keys and two tiles, where the products take 0.68,
// and 5 us of start and output for every 66 such blocks).  Short windows by
// starts and outputs, of which CTAs that stay hide a part (prompt_stay.cuh):
// 17216 packed tokens of 32 ungrouped heads, window 128, 142 to 145 us (564 MB, 84 us
// at the copy rate).
#include "few_attn.cuh"
#include "prompt_stay.cuh"

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
  return launch_prompt<kWindow>(d, rule, x, stream, nullptr, launch_stay);
}

}  // namespace spc
