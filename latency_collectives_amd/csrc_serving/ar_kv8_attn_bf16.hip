// The bfloat16 instances of the attention over the 8-bit paged cache.

#include "ar_kv8_attn.h"

namespace ard {

AttnKernel select_attn8_bf16(int head_dim, int columns) {
// rows / 16, workgroups of a compute unit, times
#define ARD_CASE(D, NQ, OCC, START, UNIT, PART) \
  if (head_dim == D && columns == NQ)           \
    return {kv8_attention<DT_BF16, D, NQ, OCC>, 256 * OCC, 16 * NQ, kAttnThreads, 12, {START, UNIT, 0.0f, PART}}
  ARD_CASE(64, 1, 3, 5.1f, 0.37f, 0.26f);
  ARD_CASE(64, 2, 2, 8.0f, 0.26f, 0.23f);
  ARD_CASE(96, 1, 2, 5.0f, 0.41f, 0.37f);
  ARD_CASE(96, 2, 2, 11.7f, 0.34f, 0.27f);
  ARD_CASE(128, 1, 2, 4.3f, 0.48f, 0.58f);
  ARD_CASE(128, 2, 2, 11.3f, 0.44f, 0.36f);
  ARD_CASE(192, 1, 2, 8.0f, 0.65f, 0.51f);
  ARD_CASE(192, 2, 1, 13.2f, 0.39f, 0.46f);
  ARD_CASE(256, 1, 1, 9.3f, 0.5f, 0.47f);
  // no 256 of 32 rows: a tile's keys and values, two of them under way, leave it too few registers
#undef ARD_CASE
  return {nullptr, 0};
}

}  // namespace ard
