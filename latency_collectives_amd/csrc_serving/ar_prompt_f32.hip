// The binary32 instances of the attention over packed prompts.

#include "ar_prompt.h"

namespace ard {

PromptKernel select_prompt_f32(int head_dim) {
#define ARD_CASE(D, NQ, SUB, OCC) \
  if (head_dim == D) return {prompt_attention<DT_F32, D, NQ, SUB, OCC>, 256 * OCC, 64 * NQ}
  ARD_CASE(64, 1, 1, 2);
  ARD_CASE(96, 1, 1, 2);
  ARD_CASE(128, 1, 1, 2);
  ARD_CASE(192, 1, 1, 1);
  ARD_CASE(256, 1, 1, 1);
#undef ARD_CASE
  return {nullptr, 0, 0};
}

}  // namespace ard
