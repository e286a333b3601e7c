// The binary32 instances of the attention over the 8-bit paged cache: queries and probabilities are
// three bfloat16 parts each, so products and sums are those of 24-bit operands.

#include "ar_kv8_attn.h"

namespace ard {

// Three products for one of bfloat16, in tiles of few rows. Two chunks of up to 2048 tokens against 12288, 16 query heads on 4: 575, 929,
// 1099, 1869 and 2522 us for heads of 64, 96, 128, 192 and 256 (240 to 270 TFLOP/s), a third to a quarter of bfloat16's rate.
AttnKernel select_attn8_f32(int head_dim, int columns) {
// rows / 16, workgroups of a compute unit, times (where there is a choice)
#define ARD_CASE(D, NQ, OCC, ...) \
  if (head_dim == D && columns == NQ) return {kv8_attention<DT_F32, D, NQ, OCC>, 256 * OCC, 16 * NQ, kAttnThreads, 12, {__VA_ARGS__}}
  ARD_CASE(64, 1, 3, 6.4f, 0.5f, 0.0f, 0.24f);
  ARD_CASE(64, 2, 2, 10.9f, 0.43f, 0.0f, 0.19f);
  ARD_CASE(96, 1, 2);
  ARD_CASE(128, 1, 2);
  ARD_CASE(192, 1, 1);
  ARD_CASE(256, 1, 1);
#undef ARD_CASE
  return {nullptr, 0};
}

}  // namespace ard
