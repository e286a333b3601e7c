// The instances of the attention over packed prompts for few rows.

#include "ar_prompt_few.h"

namespace ard {

PromptKernel select_prompt_few(int dtype, int head_dim) {
#define ARD_CASE(D) \
  if (head_dim == D) return {dtype == AR_BFLOAT16 ? prompt_attention_few<DT_BF16, D> : prompt_attention_few<DT_F32, D>, 0, 16, kAttnThreads, 0}
  ARD_CASE(64);
  ARD_CASE(96);
  ARD_CASE(128);
  ARD_CASE(192);
  ARD_CASE(256);
#undef ARD_CASE
  return {nullptr, 0, 0, 0, 0};
}

}  // namespace ard
