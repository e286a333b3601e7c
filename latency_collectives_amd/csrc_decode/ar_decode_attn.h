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
  uint32_t full;      // there: tokens from which on a tile's window counts as full
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

// Many rows a request: 32 rows for each of a workgroup's waves, if the kernel does not say otherwise.
constexpr int kRowsColumns = 2, kRowsTile = 16 * kRowsColumns * kAttnWaves;

// What a call takes of a kernel, about, in us: where it starts and ends, a unit of a run, what a unit takes besides if the
// tile is full of rows, reading back one part of a job with such a tile.
struct AttnTimes {
  float start, unit, rows, part;
};

// A kernel and the workgroups of it that fill the device's 256 compute units.
struct AttnKernel {
  void (*fn)(AttnArgs);
  int fill;
  int rows = kRowsTile;  // of a tile, where it is one for many rows
  int threads = kAttnThreads;
  // Finding a job, its queries and its end take about what twelve units of 32 tokens take while the
  // whole device reads; without them in the split, a run of many short requests ended last.
  int job_units = 12;
  AttnTimes times = {};  // where the choice goes by them
};
AttnKernel select_attn_bf16(int head_dim, int columns);
AttnKernel select_attn_f32(int head_dim, int columns);
AttnKernel select_attn_rows(int head_dim);

// The kernel for a call.
struct Choice {
  AttnKernel k;
  int rows;  // of a tile
  bool many;
};

// Tokens that a row of the table holds, below 2^31 by more than a wave looks ahead.
int64_t room_of(const ar_kv4* h, const ar_kv4_attention_args* a);

// A cache's format as the host sees it: its kernels, and the bytes of a page's heads in data and scales.
struct AttnFormat {
  AttnKernel (*bf16)(int head_dim, int columns);
  AttnKernel (*f32)(int head_dim, int columns);
  AttnKernel (*rows)(int head_dim, bool brief);  // brief: the smaller tiles, where there are two
  Choice (*choose)(const AttnFormat& f, const ar_kv4* h, const ar_kv4_attention_args* a);
  bool knows_windows;  // the split for many rows counts a full window for what it is
  int64_t (*page_bytes)(const ar_kv4* h);
  int64_t (*page_scales)(const ar_kv4* h);
};
// ar_decode_attn.hip: a handle with the workspace of these kernels, NULL on error (`name` is the entry
// point); a checked call.
ar_kv4* create_handle(const AttnFormat& f, int kv_heads, int head_dim, int page_size, const char* name);
int launch_attention(const AttnFormat& f, ar_kv4* h, const ar_kv4_attention_args* a, void* stream);

}  // namespace ard
