// The bfloat16 instances of the attention over packed prompts.

#include "ar_prompt.h"

namespace ard {

PromptKernel select_prompt_bf16(int head_dim) {
#define ARD_CASE(D, NQ, SUB, OCC) \
  if (head_dim == D) return {prompt_attention<DT_BF16, D, NQ, SUB, OCC>, 256 * OCC, 64 * NQ}
  ARD_CASE(64, 2, 2, 2);
  ARD_CASE(96, 2, 2, 2);
  ARD_CASE(128, 2, 2, 2);
  ARD_CASE(192, 2, 2, 1);
  ARD_CASE(256, 2, 1, 1);
#undef ARD_CASE
  return {nullptr, 0, 0};
}

}  // namespace ard
