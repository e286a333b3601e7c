// Host side of the 8-bit paged cache: the handle and the attention's launch, both as for the 4-bit one.

#include <algorithm>
#include <cmath>

#include "ar_kv8.h"

namespace ard {

AttnKernel select_attn8_bf16(int head_dim, int columns);
AttnKernel select_attn8_f32(int head_dim, int columns);
AttnKernel select_attn8_rows(int head_dim, bool brief);

namespace {

// What a kernel takes for a call, by the call's averages: `reqs` requests of `tokens` new ones, seeing `seen` in the mean.
double time_of(const AttnKernel& k, double reqs, double tokens, double seen, int group, int heads, int window) {
  const double each = tokens * group, tiles = std::ceil(each / k.rows), full = each / (tiles * k.rows);
  if (window > 0) seen = std::min(seen, window + static_cast<double>(k.rows) / group);
  const double units = seen / 32 + k.job_units, share = tiles * reqs * heads * units / k.fill;
  // a run of the split, and the parts that it leaves of a job
  const double run = std::max({4.0, share, std::sqrt(units)}), parts = units > run ? units / run : 0.0;
  return k.times.start + k.times.unit * std::min(run, share) + (k.times.rows * run + k.times.part * parts) * full;
}

// The kernel for a call: tiles of 16 or 32 rows with the waves on different tokens, whose parts join quickly, or of 128 to 384
// rows on the same tokens, which convert keys and values once for all of them. It is the one that takes least by its times, which
// stand beside the instances and come from every kernel's time for 1400 to 1900 calls a head size (bfloat16, 1 to 200 requests of
// 1 to 4096 tokens against 200 to 100000, 1 to 32 query heads, some with windows; binary32 400 with heads of 64). The host
// knows lengths by the tables' width alone, which a program may keep for its longest request: what counts is the product of the
// times for such lengths and for a quarter of them. How far above the best kernel the choice is in the mean, by head size (and
// at most, for nineteen of twenty), on calls that the times did not come from: 1820 with tables as wide as their lengths 0.4
// to 4.0 % (7 to 25 %), where the rule of the 4-bit cache, whose tiles have 128 rows, was 3 to 21 % (22 to 102 %); 266 four times as
// wide 0.8 to 5 %, and 6 to 9 %; 294 sixteen times as wide 9 to 16 %, and 2 to 27 %. Head of 128, 8 kv heads of 4, us with
// small tiles, tiles of 128 rows and of 384: 8 requests of 66 tokens against 8192 190, 130, 114; of 98 tokens 260, 164,
// 188; 32 of 33 tokens against 600 46, 30, 28; one of 98 against 32768 247, 128, 185; one of 400 against 2048 36, 58, 79.
Choice choose8(const AttnFormat& f, const ar_kv4* h, const ar_kv4_attention_args* a) {
  const bool bf16 = a->dtype == AR_BFLOAT16;
  const int group = a->q_heads / h->heads;
  const double reqs = std::min(a->nreq, a->ntokens), tokens = a->ntokens / reqs;
  const AttnKernel least = (bf16 ? f.bf16 : f.f32)(h->head_dim, 1);
  Choice best = {least, least.rows, false};
  if (tokens * group <= least.rows) return best;
  const double room = static_cast<double>(room_of(h, a)), own = std::min(tokens, room) / 2;
  auto time = [&](const AttnKernel& k, double length) {
    return time_of(k, reqs, tokens, std::max({length - tokens / 2, own, 1.0}), group, h->heads, a->window);
  };
  auto score = [&](const AttnKernel& k) { return time(k, room) * time(k, room / 4); };
  double lowest = score(least);
  auto look = [&](const AttnKernel& k, bool many) {
    if (k.fn == nullptr || !(score(k) < lowest)) return;
    best = {k, k.rows, many}, lowest = score(k);
  };
  look((bf16 ? f.bf16 : f.f32)(h->head_dim, 2), false);
  if (bf16) look(f.rows(h->head_dim, true), true), look(f.rows(h->head_dim, false), true);
  return best;
}

}  // namespace

static const AttnFormat kFormat8 = {select_attn8_bf16, select_attn8_f32, select_attn8_rows, choose8, true,
                                    [](const ar_kv4* h) { return int64_t(2) * h->heads * h->page_size * h->head_dim; },
                                    [](const ar_kv4* h) { return int64_t(2) * h->heads * (h->page_size / kBlock); }};

}  // namespace ard

extern "C" {

ar_kv8* ar_kv8_create(int kv_heads, int head_dim, int page_size) {
  return static_cast<ar_kv8*>(ard::create_handle(ard::kFormat8, kv_heads, head_dim, page_size, "ar_kv8_create"));
}

void ar_kv8_destroy(ar_kv8* h) { ar_kv4_destroy(h); }

int ar_kv8_attention(ar_kv8* h, const ar_kv8_attention_args* a, void* stream) {
  return ard::launch_attention(ard::kFormat8, h, a, stream);
}

}  // extern "C"
