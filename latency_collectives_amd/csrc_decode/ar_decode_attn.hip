// Host side of the attention over the 4-bit paged cache: the handle and the launch.

#include <algorithm>
#include <cmath>
#include <new>

#include "ar_decode_attn.h"

namespace {

// The kernel for a call. Tiles of 16 or 32 rows, four waves on different tokens: short jobs, whose
// parts join quickly. Tiles of 128 rows, waves on different rows: values are converted once for all
// of them, but a job is four times as long and so is its join, so they pay where the tiles alone
// fill the device's 512 places and have some tokens to read, or where the tokens behind them are many.
// Small tiles against large, head_dim 128, 4 kv heads of 8 query heads, 4096 tokens: 8 requests of 512
// rows 59 and 87 us, of 1024 103 and 112, of 2048 (512 tiles) 190 and 183, of 4096 373 and 307, of 16384
// 1492 and 915; one of 4096 rows and 16384 tokens 188 and 182, of 8192 rows 349 and 302; head_dim 64, 552
// tiles of one prompt, 786 tokens 62 and 46. Binary32, three products for one, stays with the small
// tiles. The tokens that the host knows are the tables' width, and these are times of tables as wide
// as the longest request. Wider ones move the second rule's border and not the work: with room for
// 131072 tokens the 8 requests of 512 rows take the large tiles' 87 us, one of 1004 rows and 1711
// tokens 53 for 29. Tables no wider than the step's longest request avoid it.
constexpr int64_t kManyTiles = 512, kManyUnits = 1 << 16, kFewTiles = 128;

// Tokens that a row of the table holds, below 2^31 by more than a wave looks ahead.
int64_t room_of(const ar_kv4* h, const ar_kv4_attention_args* a) {
  return std::min<int64_t>(static_cast<int64_t>(a->table_width) << h->page_shift, 0x7FF00000);
}

struct Choice {
  ard::AttnKernel k;
  int rows;  // of a tile
  bool many;
};

Choice choose(const ar_kv4* h, const ar_kv4_attention_args* a) {
  const int64_t rows = static_cast<int64_t>(a->ntokens) * (a->q_heads / h->heads);
  const int64_t each = (rows + a->nreq - 1) / a->nreq;
  const bool bf16 = a->dtype == AR_BFLOAT16;
  if (bf16 && each > 128) {
    const int large = ard::kRowsTile;
    const int64_t tiles = (each + large - 1) / large * std::min(a->nreq, a->ntokens) * h->heads;
    const int64_t tokens = room_of(h, a);
    const int64_t units = (a->window > 0 ? std::min<int64_t>(tokens, a->window) : tokens) / 32 + 1;
    if ((tiles >= kManyTiles && units >= 16) || tiles * units >= kManyUnits)
      return {ard::select_attn_rows(h->head_dim), large, true};
  }
  // Twice the rows for one reading of the cache, where enough tiles are left for the device (bfloat16,
  // head_dim 128, 4 kv heads, 16 rows a tile and 32: 64 requests of 64 rows, 2048 tokens 55 and
  // 30 us; one of 32 rows, 4096 tokens 11.8 and 15.7). Binary32 gains from it at head_dim 64 only.
  const int64_t tiles = (each + 31) / 32 * std::min(a->nreq, a->ntokens) * h->heads;
  const int columns = each > 16 && tiles >= kFewTiles && (bf16 || h->head_dim == 64) ? 2 : 1;
  return {bf16 ? ard::select_attn_bf16(h->head_dim, columns) : ard::select_attn_f32(h->head_dim, columns), 16 * columns,
          false};
}

// Partial results of a launch: two slots a workgroup (the job it ends, the job it begins), each
// `rows` rows of head_dim sums and a {max, sum} pair.
size_t part_bytes(int runs, int rows, int head_dim) {
  return size_t(2) * runs * rows * (head_dim + 2) * sizeof(float);
}

constexpr int kMostRuns = 1024;  // at least every kernel's `fill`
constexpr size_t kArrivedBytes = kMostRuns * sizeof(uint32_t);

// Finding a job, its queries and its end take about what twelve units of 32 tokens take while the
// whole device reads; without them in the split, a run of many short requests ended last.
constexpr int kJobUnits = 12;

}  // namespace

extern "C" {

ar_kv4* ar_kv4_create(int kv_heads, int head_dim, int page_size) {
  if (kv_heads < 1 || kv_heads > 1024) {
    ar_fail(AR_EINVAL, "kv_heads must be in [1, 1024], got %d", kv_heads);
    return nullptr;
  }
  if (head_dim != 64 && head_dim != 96 && head_dim != 128 && head_dim != 192 && head_dim != 256) {
    ar_fail(AR_ENOTSUP, "head_dim must be 64, 96, 128, 192 or 256, got %d", head_dim);
    return nullptr;
  }
  if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0) {
    ar_fail(AR_EINVAL, "page_size must be a power of two in [16, 1024], got %d", page_size);
    return nullptr;
  }
  ar_kv4* h = new (std::nothrow) ar_kv4;
  if (h == nullptr) {
    ar_fail(AR_ENORES, "out of host memory");
    return nullptr;
  }
  *h = ar_kv4{kv_heads, head_dim, page_size, __builtin_ctz(page_size), -1, nullptr, 0};
  for (int n = 1; n <= 2; ++n)
    for (const ard::AttnKernel& k : {ard::select_attn_bf16(head_dim, n), ard::select_attn_f32(head_dim, n)})
      h->work_bytes = std::max(h->work_bytes, part_bytes(k.fill, 16 * n, head_dim));
  h->work_bytes = std::max(h->work_bytes, part_bytes(ard::select_attn_rows(head_dim).fill,
                                                     ard::kRowsTile, head_dim));
  int devices = 0;
  if (hipGetDeviceCount(&devices) != hipSuccess || devices == 0) {
    (void)hipGetLastError();
    return h;
  }
  hipError_t e = hipGetDevice(&h->device);
  if (e == hipSuccess) e = hipMalloc(&h->work, h->work_bytes + kArrivedBytes);
  if (e == hipSuccess) e = hipMemset(static_cast<uint8_t*>(h->work) + h->work_bytes, 0, kArrivedBytes);
  if (e == hipSuccess) e = hipDeviceSynchronize();
  if (e != hipSuccess) {
    ar_fail_hip(e, "the workspace of ar_kv4_create");
    if (h->work != nullptr) (void)hipFree(h->work);
    delete h;
    return nullptr;
  }
  return h;
}

void ar_kv4_destroy(ar_kv4* h) {
  if (h == nullptr) return;
  if (h->work != nullptr) {
    int current = h->device;
    (void)hipGetDevice(&current);
    if (current != h->device) (void)hipSetDevice(h->device);
    (void)hipDeviceSynchronize();
    (void)hipFree(h->work);
    if (current != h->device) (void)hipSetDevice(current);
  }
  delete h;
}

int ar_kv4_attention(ar_kv4* h, const ar_kv4_attention_args* a, void* stream) {
  using namespace ard;
  if (int rc = check_handle(h)) return rc;
  if (a == nullptr) return ar_fail(AR_EINVAL, "null arguments");
  if (int rc = check_dtype(a->dtype)) return rc;
  if (a->ntokens < 0 || a->nreq < 0 || a->table_width < 0) return ar_fail(AR_EINVAL, "negative size");
  if (a->q_heads < 1 || a->q_heads % h->heads != 0)
    return ar_fail(AR_EINVAL, "q_heads must be a multiple of the %d kv heads, got %d", h->heads, a->q_heads);
  if (a->q_heads > 65536) return ar_fail(AR_ETOOBIG, "too many heads");
  if (a->window < 0) return ar_fail(AR_EINVAL, "window must not be negative, got %d", a->window);
  const float scale_log2 = static_cast<float>(a->scale * 1.4426950408889634);
  if (!std::isfinite(scale_log2)) return ar_fail(AR_EINVAL, "scale must be finite in binary32, as its product with log2(e)");
  if (int rc = check_cache(a->data, a->scales, a->num_pages)) return rc;
  if (a->table_stride < a->table_width) return ar_fail(AR_EINVAL, "table_stride is below table_width");
  if (a->ntokens == 0 || a->nreq == 0) return AR_OK;
  if (a->q == nullptr || a->out == nullptr) return ar_fail(AR_EINVAL, "null q or out");
  if (a->kv_len == nullptr || a->q_start == nullptr || (a->table_width > 0 && a->table == nullptr))
    return ar_fail(AR_EINVAL, "null request buffer");
  const int64_t unit = a->dtype == AR_BFLOAT16 ? 8 : 4;
  if (!aligned(a->q, 16) || !aligned(a->out, 16) || a->q_token % unit != 0 || a->q_head % unit != 0 ||
      a->o_token % unit != 0 || a->o_head % unit != 0)
    return ar_fail(AR_EINVAL, "q and out: addresses and strides must be multiples of 16 bytes");
  if (a->q_token < 0 || a->q_head < 0 || a->o_token < 0 || a->o_head < 0)
    return ar_fail(AR_EINVAL, "negative stride");
  // Rows of a kv head, and a unit of every job beside what its start and end count for, in 31 bits.
  const int64_t all_rows = static_cast<int64_t>(a->ntokens) * (a->q_heads / h->heads);
  if (all_rows > 0x7FFFFFFF) return ar_fail(AR_ETOOBIG, "too many rows");
  const Choice choice = choose(h, a);
  const AttnKernel& k = choice.k;
  if (k.fn == nullptr) return ar_fail(AR_ENOTSUP, "no kernel for head_dim %d", h->head_dim);
  const int rows_per_tile = choice.rows;
  const int64_t tiles = all_rows / rows_per_tile + std::min(a->nreq, a->ntokens), jobs = tiles * h->heads;
  if (tiles * rows_per_tile > 0x7FFFFFFF || jobs * (1 + kJobUnits) > 0x7FFFFFFF)
    return ar_fail(AR_ETOOBIG, "too many rows");
  if (h->work == nullptr) return ar_fail(AR_EHIP, "the handle was created without a GPU");
  int device = -1;
  AR_HIP(hipGetDevice(&device));
  if (device != h->device)
    return ar_fail(AR_EINVAL, "the handle was created on GPU %d, the current one is %d", h->device, device);

  AttnArgs args;
  args.a = *a;
  args.cache = Cache{const_cast<uint8_t*>(a->data), const_cast<uint8_t*>(a->scales), a->num_pages,
                     h->heads, h->page_shift};
  args.group = a->q_heads / h->heads;
  args.per_group = 1.0f / args.group;
  args.page_bytes = static_cast<int64_t>(h->heads) * h->page_size * h->head_dim;
  args.page_scales = static_cast<int64_t>(h->heads) * 2 * h->page_size * (h->head_dim / 32);
  args.scale_log2 = scale_log2;
  args.q_sign = 0;
  if (choice.many) {
    if (a->scale < 0) args.q_sign = 0x80008000u;
    // not zero: a masked score's infinity times it has to stay one
    args.scale_log2 = std::max(std::fabs(args.scale_log2), 1e-38f);
  }
  args.part = static_cast<uint8_t*>(h->work);
  args.part_bytes = static_cast<uint32_t>(part_bytes(k.fill, choice.rows, h->head_dim));
  args.stats_at = 2u * k.fill * choice.rows * h->head_dim * 4;
  args.arrived = reinterpret_cast<uint32_t*>(args.part + h->work_bytes);
  // As many workgroups as the device holds at once, of at least four units of 32 tokens each: fewer
  // where the requests cannot have more. Larger units where 32-bit sums of them could overflow: a unit
  // of 2^31 tokens is the last, which leaves each job the one that the check above counts.
  const int64_t room = room_of(h, a);
  int64_t seen = room;
  // what a tile's rows see with a window: their tokens and the start's rounding down to 32
  if (a->window > 0) seen = std::min<int64_t>(seen, static_cast<int64_t>(a->window) + rows_per_tile / args.group + 33);
  args.room = static_cast<int>(room);
  args.most_seen = static_cast<uint32_t>(seen);
  args.unit_shift = 5;
  const auto span = [&] { return ((seen + (int64_t(1) << args.unit_shift) - 1) >> args.unit_shift) + kJobUnits; };
  while (span() * jobs > 0x7FFFFFFF) ++args.unit_shift;
  args.unit = 1u << args.unit_shift;
  args.tile_shift = args.unit_shift - 5;
  args.tile_tokens = (rows_per_tile - 1) / args.group + 1;
  args.job_units = kJobUnits;
  const int64_t runs = (jobs * span() + kAttnWaves - 1) / kAttnWaves;
  int64_t grid = std::min<int64_t>(k.fill, runs);
  if (choice.many) grid = (grid + 7) & ~7;  // the same number for every XCD
  args.runs = static_cast<uint32_t>(grid);
  hipLaunchKernelGGL(k.fn, dim3(static_cast<unsigned>(grid)), dim3(kAttnThreads), 0,
                     static_cast<hipStream_t>(stream), args);
  AR_HIP(hipGetLastError());
  return AR_OK;
}

}  // extern "C"
