// Host side of the attention over packed prompts: the handle and the launch.

#include "ar_prompt.h"

#include <algorithm>
#include <cmath>
#include <new>

// The handle behind ar_prompt.
struct ar_prompt {
  int heads, head_dim;
  int device;      // where it was created, -1 without a GPU
  void* work;      // partial results, then arrival counters; NULL without a GPU
  size_t work_bytes;
};

namespace ard {
namespace {

// Partial results of a launch: two slots a workgroup (the job it ends, the job it begins), each
// `rows` rows of head_dim sums and a {max, sum} pair.
size_t prompt_part_bytes(const PromptKernel& k, int head_dim) {
  return size_t(2) * k.fill * k.rows * (head_dim + 2) * sizeof(float);
}

constexpr size_t kPromptArrived = 1024 * sizeof(uint32_t);  // at least every kernel's `fill`

// Few rows: a workgroup for 16 rows and a kv head, which takes its units without a share for others. As long as jobs times
// units, with kFewJobUnits for a job's start and end, times head_dim stay below kFewWork, half as much again for
// binary32, whose other kernels take longer to start. us with few rows' kernel and with the others (and that product, in
// 2^20), head of 128, 8 query heads on one kv head: one prompt of 301 tokens (0.3) 7.9 and 16.2, of 1000 (1.7) 21.0 and 35.4, of 1500
// (3.3) 36.2 and 39.8, of 1700 (4.0) 42.4 and 40.2; 32 heads on 8: one of 500 (2.4) 21.9 and 25.2, of 600 (3.2) 29.3 and 27.1, of
// 800 (4.9) 42.8 and 30.7, 16 of up to 100 (2.8) 15.6 and 16.9. Head of 64, 32 on 8, 800 tokens (2.4) 25.8 and 22.5; of 256, 8 on
// 8, 20 of up to 100 (2.0) 22.5 and 22.1, 8 on one, 900 tokens (3.0) 30.5 and 54.6, 1400 (5.8) 62.0 and 57.3. Binary32, 128: 1700
// tokens (4.0) 74.5 and 102.6, 32 heads, 800 (4.9) 81.5 and 80.7. With the rule below, on 4100 random calls (one long prompt
// among short ones in a quarter of them) the choice takes 0.7 to 4 % longer than the best kernel in the mean, by type and head, 4
// to 17 % at nineteen of twenty; 2.8 times at worst (binary32, head of 192, 280 prompts of a token or eight, 64 heads on 8).
constexpr int kFewJobUnits = 12, kFewWork = 3 << 20;

// Large tiles: where every workgroup gets so many units of its tile's rows. us without and with them, head of 128: one prompt of
// 4000 tokens, 8 heads on one (20), 65 and 76, of 6000 (46) 104 and 107, of 8000 (82) 163 and 146; eight of up to 2000, 32 on 8
// (48), 168 and 153.
constexpr int kLargeUnits = 40;

}  // namespace
}  // namespace ard

extern "C" {

ar_prompt* ar_prompt_create(int kv_heads, int head_dim) {
  using namespace ard;
  if (kv_heads < 1 || kv_heads > 1024) {
    ar_fail(AR_EINVAL, "kv_heads must be in [1, 1024], got %d", kv_heads);
    return nullptr;
  }
  const PromptKernel all[] = {select_prompt_bf16(head_dim, false), select_prompt_bf16(head_dim, true), select_prompt_f32(head_dim)};
  size_t work_bytes = 0;
  for (const PromptKernel& k : all) work_bytes = std::max(work_bytes, k.fn == nullptr ? 0 : prompt_part_bytes(k, head_dim));
  if (work_bytes == 0) {
    ar_fail(AR_ENOTSUP, "head_dim must be 64, 96, 128, 192 or 256, got %d", head_dim);
    return nullptr;
  }
  ar_prompt* h = new (std::nothrow) ar_prompt;
  if (h == nullptr) {
    ar_fail(AR_ENORES, "out of host memory");
    return nullptr;
  }
  *h = ar_prompt{kv_heads, head_dim, -1, nullptr, work_bytes};
  int devices = 0;
  if (hipGetDeviceCount(&devices) != hipSuccess || devices == 0) {
    (void)hipGetLastError();
    return h;
  }
  hipError_t e = hipGetDevice(&h->device);
  if (e == hipSuccess) e = hipMalloc(&h->work, h->work_bytes + kPromptArrived);
  if (e == hipSuccess) e = hipMemset(static_cast<uint8_t*>(h->work) + h->work_bytes, 0, kPromptArrived);
  if (e == hipSuccess) e = hipDeviceSynchronize();
  if (e != hipSuccess) {
    ar_fail_hip(e, "ar_prompt_create");
    if (h->work != nullptr) (void)hipFree(h->work);
    delete h;
    return nullptr;
  }
  return h;
}

void ar_prompt_destroy(ar_prompt* h) {
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

int ar_prompt_attention(ar_prompt* h, const ar_prompt_attention_args* a, void* stream) {
  using namespace ard;
  if (h == nullptr) return ar_fail(AR_EINVAL, "null handle");
  if (a == nullptr) return ar_fail(AR_EINVAL, "null arguments");
  if (int rc = check_dtype(a->dtype)) return rc;
  if (a->ntokens < 0 || a->nreq < 0) return ar_fail(AR_EINVAL, "negative size");
  if (a->q_heads < 1 || a->q_heads % h->heads != 0)
    return ar_fail(AR_EINVAL, "q_heads must be a multiple of the %d kv heads, got %d", h->heads, a->q_heads);
  if (a->q_heads > 65536) return ar_fail(AR_ETOOBIG, "too many heads");
  if (a->window < 0) return ar_fail(AR_EINVAL, "window must not be negative, got %d", a->window);
  const float scale_log2 = static_cast<float>(a->scale * 1.4426950408889634);
  if (!std::isfinite(scale_log2)) return ar_fail(AR_EINVAL, "scale must be finite in binary32, as its product with log2(e)");
  if (a->ntokens == 0 || a->nreq == 0) return AR_OK;
  if (a->nreq > INT32_MAX - 128) return ar_fail(AR_ETOOBIG, "too many requests");
  if (a->q == nullptr || a->k == nullptr || a->v == nullptr || a->out == nullptr) return ar_fail(AR_EINVAL, "null q, k, v or out");
  if (a->q_start == nullptr) return ar_fail(AR_EINVAL, "null q_start");
  const bool bf16 = a->dtype == AR_BFLOAT16;
  const int64_t unit = bf16 ? 8 : 4, bytes = bf16 ? 2 : 4;
  for (const void* p : {a->q, a->k, a->v, static_cast<const void*>(a->out)})
    if (!aligned(p, 16)) return ar_fail(AR_EINVAL, "q, k, v and out: addresses must be multiples of 16 bytes");
  for (int64_t s : {a->q_token, a->q_head, a->k_token, a->k_head, a->v_token, a->v_head, a->o_token, a->o_head}) {
    if (s % unit != 0) return ar_fail(AR_EINVAL, "q, k, v and out: strides must be multiples of 16 bytes");
    if (s < 0) return ar_fail(AR_EINVAL, "negative stride");
  }
  if (std::max(a->k_token, a->v_token) > kMostStride / bytes) return ar_fail(AR_ETOOBIG, "a token's keys or values are more than 2^23 bytes apart");
  // Rows of a kv head, and a unit of every job beside what its start and end count for, in 31 bits.
  const int group = a->q_heads / h->heads;
  const int64_t all_rows = static_cast<int64_t>(a->ntokens) * group;
  if (all_rows > 0x7FFFFFFF) return ar_fail(AR_ETOOBIG, "too many rows");
  // The kernel, by the tiles, and the units of 32 tokens that their rows see, if prompts are alike.
  const int prompts = std::min(a->nreq, a->ntokens);
  int64_t sees = a->ntokens / prompts;
  sees = a->window > 0 ? std::min<int64_t>(sees / 2, a->window) : sees / 2;
  const int64_t units = sees / 32 + 1;
  PromptKernel k = select_prompt_few(a->dtype, h->head_dim);
  int64_t tiles = all_rows / k.rows + prompts, jobs = tiles * h->heads;
  const int64_t alike = (all_rows / prompts + k.rows - 1) / k.rows * prompts * h->heads;
  const bool few = alike * (units + kFewJobUnits) * h->head_dim <= (bf16 ? kFewWork : kFewWork / 2 * 3);
  if (!few) {
    k = bf16 ? select_prompt_bf16(h->head_dim, true) : select_prompt_f32(h->head_dim);
    if (bf16 && all_rows * h->heads / k.rows * units < kLargeUnits * k.fill) k = select_prompt_bf16(h->head_dim, false);
    tiles = all_rows / k.rows + prompts, jobs = tiles * h->heads;
    if (tiles * k.rows > 0x7FFFFFFF || jobs * (1 + k.job_units) > 0x7FFFFFFF) return ar_fail(AR_ETOOBIG, "too many rows");
  }
  if (h->work == nullptr) return ar_fail(AR_EHIP, "the handle was created without a GPU");
  int device = -1;
  AR_HIP(hipGetDevice(&device));
  if (device != h->device)
    return ar_fail(AR_EINVAL, "the handle was created on GPU %d, the current one is %d", h->device, device);

  PromptArgs args;
  args.a = *a;
  args.cache.heads = h->heads;
  args.group = group;
  args.per_group = 1.0f / group;
  args.scale_log2 = scale_log2;
  args.q_sign = 0;
  if (bf16) {
    if (a->scale < 0) args.q_sign = 0x80008000u;
    // not zero: a masked score's infinity times it has to stay one
    args.scale_log2 = std::max(std::fabs(args.scale_log2), 1e-38f);
  }
  if (few) {
    args.runs = static_cast<uint32_t>(tiles);
    hipLaunchKernelGGL(k.fn, dim3(static_cast<unsigned>(tiles), h->heads), dim3(k.threads), 0, static_cast<hipStream_t>(stream), args);
    AR_HIP(hipGetLastError());
    return AR_OK;
  }
  args.part = static_cast<uint8_t*>(h->work);
  args.part_bytes = static_cast<uint32_t>(prompt_part_bytes(k, h->head_dim));
  args.stats_at = 2u * k.fill * k.rows * h->head_dim * 4;
  args.arrived = reinterpret_cast<uint32_t*>(args.part + h->work_bytes);
  args.tile_tokens = (k.rows - 1) / group + 1;
  int64_t seen = a->ntokens;
  // what a tile's rows see with a window: their tokens and the start's rounding down to 32
  if (a->window > 0) seen = std::min<int64_t>(seen, static_cast<int64_t>(a->window) + k.rows / group + 33);
  args.most_seen = static_cast<uint32_t>(seen);
  // Larger units where 32-bit sums of them could overflow.
  args.unit_shift = 5;
  args.job_units = k.job_units;
  const auto span = [&] { return ((seen + (int64_t(1) << args.unit_shift) - 1) >> args.unit_shift) + k.job_units; };
  while (span() * jobs > 0x7FFFFFFF) ++args.unit_shift;
  args.unit = 1u << args.unit_shift;
  args.tile_shift = args.unit_shift - 5;
  // As many workgroups as the device holds at once, fewer where there cannot be a round of units for each;
  // the same number for every XCD.
  const int64_t runs = (jobs * span() + kAttnWaves - 1) / kAttnWaves;
  const int64_t grid = (std::min<int64_t>(k.fill, runs) + 7) & ~int64_t(7);
  args.runs = static_cast<uint32_t>(grid);
  hipLaunchKernelGGL(k.fn, dim3(static_cast<unsigned>(grid)), dim3(k.threads), 0, static_cast<hipStream_t>(stream), args);
  AR_HIP(hipGetLastError());
  return AR_OK;
}

}  // extern "C"
