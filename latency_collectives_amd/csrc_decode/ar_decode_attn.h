// Arguments and dispatch of the attention over the 4-bit paged cache.
#pragma once

#include "ar_decode.h"

namespace ard {

struct AttnArgs {
  ar_kv4_attention_args a;
  Cache cache;
  int64_t page_bytes, page_scales;  // of a page's heads, in data and scales
  int group;          // query heads of a kv head
  float per_group;    // 1 / group
  int room;           // tokens that a row of the table holds
  // The work split: units of `unit` tokens (32 << tile_shift), of which a row sees at most
  // most_seen; at most `runs` runs.
  uint32_t most_seen, unit, runs;
  int unit_shift, tile_shift;
  int job_units;      // what starting and ending a job costs, in units
  float scale_log2;   // scale * log2(e); its absolute value for the kernel of many rows
  uint32_t q_sign;    // there: its sign, on two bfloat16
  int tile_tokens;    // there: tokens that a tile of rows may touch
  uint8_t* part;      // partial sums [slot][row][head_dim], then {max, sum} [slot][row]
  uint32_t part_bytes;
  uint32_t stats_at;  // byte offset of the {max, sum} pairs in `part`
  uint32_t* arrived;  // [workgroup of a job's first part]: parts done
};

// Rows (tokens x heads of a group) of a query tile are 16 * columns.
constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = kAttnThreads / 64;

// A kernel and the workgroups of it that fill the device's 256 compute units.
struct AttnKernel {
  void (*fn)(AttnArgs);
  int fill;
};
AttnKernel select_attn_bf16(int head_dim, int columns);
AttnKernel select_attn_f32(int head_dim, int columns);
// Many rows a request: 32 rows for each of a workgroup's waves.
constexpr int kRowsColumns = 2, kRowsTile = 16 * kRowsColumns * kAttnWaves;
AttnKernel select_attn_rows(int head_dim);

}  // namespace ard
