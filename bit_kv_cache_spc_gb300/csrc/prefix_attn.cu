// The attention of sequences that share a prefix: every query sees all of the
// prefix, whose keys and values are stored once, and of its own sequence's keys
// those that are not behind it.  The kernel of prompt_attn.cuh, walking over the
// prefix's blocks and then over the sequence's; or, where the sequences have few
// rows, over the prefix with the rows of all of them together, and then over
// each one's own keys (single tokens with few_attn.cuh's kernel).
// 64 single tokens of 32 and 8 heads behind 32768 keys, up to 1024 of their own
// (276 MB, 41 us at the copy rate): 62 to 65 us, against 1035 with the prefix
// walked for each.  17 prompts of up to 77 tokens, 32 ungrouped heads, behind
// 8011 keys (81 GFLOP, 43 us at the burst rate): 104 to 108 us, against 315.
// Four of up to 2048 tokens behind 16384 keys, one by one (1.02 TFLOP, 537 us):
// 624 to 676 us.  64 batched prompts of 17 tokens, 32 and 8 heads, behind 8192
// keys, each of which walks over these: 274 us, packed 107 (of 16 tokens 106 and
// 106).
#include "few_attn.cuh"

namespace spc {

cudaError_t prefix_fault_word(void** word) { return cudaGetSymbolAddress(word, prompt_device_fault); }

size_t prefix_workspace_bytes(const spc_prompt_dims* d, const spc_prefix* p) {
  PromptRule rule;
  rule.prefix = p->tokens;
  return prompt_bytes(d, rule);
}

int32_t prefix_together(const spc_prompt_dims* d, const spc_prefix* p, bool placed) {
  PromptRule rule;
  rule.prefix = p->tokens;
  const PromptGrid g = together_grid(d, rule);
  return !taken_together(d, g, placed) ? 0 : g.mixed ? 2 : 1;
}

spc_status launch_prefix_attn(const spc_prompt_dims* d, const spc_prefix* p, const uint16_t* q, const uint16_t* pk,
                              const uint16_t* pv, const int32_t* p_len, const uint16_t* k, const uint16_t* v,
                              const int32_t* q_begin, const int32_t* q_len, const int32_t* k_begin,
                              const int32_t* k_len, uint16_t* o, float* lse, void* ws, cudaStream_t stream) {
  PromptRule rule;
  rule.prefix = p->tokens;
  return launch_prompt<kPrefix>(d, rule, {q, k, v, q_begin, q_len, k_begin, k_len, o, lse, ws, pk, pv, p_len, p}, stream,
                                launch_few<true>);
}

}  // namespace spc
