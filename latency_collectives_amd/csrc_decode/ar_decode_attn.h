// Arguments and dispatch of the attention over the 4-bit paged cache.
#pragma once

#include "ar_decode.h"

namespace ard {

struct AttnArgs {
  ar_kv4_attention_args a;
  Cache cache;
  int group;          // query heads of a kv head
  int target_shift;   // the work is cut into about 2^target_shift items
  float scale_log2;   // scale * log2(e)
  uint8_t* part;      // partial sums [slot][row][head_dim], then {max, sum} [slot][row]
  uint32_t part_bytes;
  uint32_t stats_at;  // byte offset of the {max, sum} pairs in `part`
  uint32_t* arrived;  // [slot of a job's first part]: parts done
};

// Rows (tokens x heads of a group) of a query tile are 16 * columns.
constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = kAttnThreads / 64;

typedef void (*attn_fn)(AttnArgs);
attn_fn select_attn_bf16(int head_dim, int columns);
attn_fn select_attn_f32(int head_dim, int columns);

// Items a launch is cut into (before rounding up per job), as a power of two: what fills the
// device's 256 compute units at the occupancy of the variant.
constexpr int target_shift(int columns) { return columns == 1 ? 10 : 9; }

}  // namespace ard
