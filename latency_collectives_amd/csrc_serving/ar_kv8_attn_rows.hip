// The instances of the attention over the 8-bit paged cache for many rows a request.

#include "ar_kv8_attn_rows.h"

namespace ard {

// Two chunks of up to 2048 tokens against 12288, TFLOP/s, 16 query heads on 4 (128 with 32 on 8: 1030 to 1050), and one layout beside:
//   64    8 waves of 32 rows, twice a compute unit   770    (8 of 16, twice: 697)
//   96    12 of 32     769    (8 of 16, twice: 657)
//   128   12 of 32     952    (8 of 32: 878; 8 of 16, twice: 810)
//   192   12 of 16     905    (8 of 32: 900)
//   256   12 of 16     834    (8 of 16: 732)
// Tiles of 12 waves of 32 rows are large for requests of few rows or tokens: heads of 96 and 128 have 8 waves of 16 beside.
constexpr int kJobUnits = 8;  // what starting and ending a job costs; 4 and 12 are within 1% mostly

AttnKernel select_attn8_rows(int head_dim, bool brief) {
// rows / 16 of a wave, waves of a workgroup, units of a round, workgroups of a compute unit, times
#define ARD_CASE(D, NQ, WAVES, SUB, OCC, START, UNIT, ROWS, PART)                                                                    \
  if (head_dim == D)                                                                                                                 \
    return {kv8_attention_rows<D, NQ, WAVES, SUB, OCC * WAVES / 4>, 256 * OCC, 16 * NQ * WAVES, 64 * WAVES, kJobUnits,               \
            {START, UNIT, ROWS, PART}}
  if (brief) {
    ARD_CASE(96, 1, 8, 2, 2, 11.0f, 0.73f, 0.36f, 5.2f);
    ARD_CASE(128, 1, 8, 2, 2, 13.4f, 0.6f, 0.46f, 2.9f);
  }
  ARD_CASE(64, 2, 8, 4, 2, 12.2f, 0.42f, 0.67f, 6.0f);
  ARD_CASE(96, 2, 12, 3, 1, 18.4f, 0.65f, 0.66f, 3.5f);
  ARD_CASE(128, 2, 12, 3, 1, 11.7f, 0.49f, 0.8f, 8.5f);
  ARD_CASE(192, 1, 12, 2, 1, 10.5f, 0.55f, 0.45f, 6.3f);
  ARD_CASE(256, 1, 12, 1, 1, 24.3f, 0.92f, 0.94f, 3.9f);
#undef ARD_CASE
  return {nullptr, 0};
}

}  // namespace ard
