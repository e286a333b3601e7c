// The bfloat16 instances of the attention over the 8-bit paged cache.

#include "ar_kv8_attn.h"

namespace ard {

AttnKernel select_attn8_bf16(int head_dim, int columns) {
#define ARD_CASE(D, NQ, OCC) \
  if (head_dim == D && columns == NQ) return {kv8_attention<DT_BF16, D, NQ, OCC>, 256 * OCC}
  ARD_CASE(64, 1, 3);
  ARD_CASE(64, 2, 2);
  ARD_CASE(96, 1, 2);
  ARD_CASE(96, 2, 2);
  ARD_CASE(128, 1, 2);
  ARD_CASE(128, 2, 2);
  ARD_CASE(192, 1, 2);
  ARD_CASE(192, 2, 1);
  ARD_CASE(256, 1, 1);
  // no 256 of 32 rows: a tile's keys and values, two of them under way, leave it too few registers
#undef ARD_CASE
  return {nullptr, 0};
}

}  // namespace ard
