// The binary32 instances of the attention over the 4-bit paged cache: queries and probabilities
// are three bfloat16 parts each, so products and sums are those of 24-bit operands.

#include "ar_decode_attn_impl.h"

namespace ard {

AttnKernel select_attn_f32(int head_dim, int columns) {
#define ARD_CASE(D, NQ, OCC) \
  if (head_dim == D && columns == NQ) return {kv4_attention<DT_F32, D, NQ, OCC>, 256 * OCC}
  ARD_CASE(64, 1, 3);
  ARD_CASE(64, 2, 2);
  ARD_CASE(96, 1, 2);
  ARD_CASE(128, 1, 2);
  ARD_CASE(192, 1, 1);
  ARD_CASE(256, 1, 1);
#undef ARD_CASE
  return {nullptr, 0};
}

}  // namespace ard
