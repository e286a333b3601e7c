// The instances of the attention over the 8-bit paged cache for many rows a request.

#include "ar_kv8_attn_rows.h"

namespace ard {

AttnKernel select_attn8_rows(int head_dim) {
#define ARD_CASE(D, OCC) \
  if (head_dim == D) return {kv8_attention_rows<D, kRowsColumns, OCC>, 256 * OCC}
  ARD_CASE(64, 2);
  ARD_CASE(96, 2);
  ARD_CASE(128, 2);
  ARD_CASE(192, 1);
  ARD_CASE(256, 1);
#undef ARD_CASE
  return {nullptr, 0};
}

}  // namespace ard
