// The instances of the attention over the 8-bit paged cache for many rows a request.

#include "ar_kv8_attn_rows.h"

namespace ard {

// Two chunks of up to 2048 tokens against 12288, TFLOP/s (16 query heads on 4; 128: 32 on 8), and one layout beside:
//   64    8 waves of 32 rows, twice a compute unit   759    (8 of 16, twice: 684)
//   96    12 of 32     747    (8 of 16, twice: 654)
//   128   12 of 32     957    (8 of 32: 864; 8 of 16, twice: 846)
//   192   12 of 16     831    (8 of 32: 798)
//   256   12 of 16     831    (8 of 16: 718)
// Rows that see few tokens would rather have small tiles, 8 waves of 16 rows, where the large ones are 12 waves' (128, 16 heads on
// 4, us): 32 chunks of 256 tokens against 512 88 and 80, 16 against 2048 126 and 117, against 4096 190 and 191; four of 2048
// with a window of 1000 136 and 96, of 4000 324 and 308. A head of 64 loses what windows cost it by them (58.7 and 67.5).
constexpr int kJobUnits = 8;  // what starting and ending a job costs; 4 and 12 are within 1% mostly

AttnKernel select_attn8_rows(int head_dim, bool brief) {
// rows / 16 of a wave, waves of a workgroup, units of a round, workgroups of a compute unit
#define ARD_CASE(D, NQ, WAVES, SUB, OCC) \
  if (head_dim == D) return {kv8_attention_rows<D, NQ, WAVES, SUB, OCC * WAVES / 4>, 256 * OCC, 16 * NQ * WAVES, 64 * WAVES, kJobUnits}
  if (brief) {
    ARD_CASE(96, 1, 8, 2, 2);
    ARD_CASE(128, 1, 8, 2, 2);
  }
  ARD_CASE(64, 2, 8, 4, 2);
  ARD_CASE(96, 2, 12, 3, 1);
  ARD_CASE(128, 2, 12, 3, 1);
  ARD_CASE(192, 1, 12, 2, 1);
  ARD_CASE(256, 1, 12, 1, 1);
#undef ARD_CASE
  return {nullptr, 0};
}

}  // namespace ard
