// ar_page_tables: block tables, slots and positions of a decode step from the requests' lengths.
//
// Two prefix sums over the requests (pages taken, tokens brought) decide everything; the rest is
// one value a token or a new page. Every workgroup computes the sums of all requests for itself
// (a request's share is 8 bytes, 4096 requests a few microseconds) and then fills its part of the
// outputs, so one launch does a step and no workgroup waits for another.

#include "ar_decode.h"

namespace ard {

constexpr int kMaxRequests = 4096;
constexpr int kTableThreads = 1024;
constexpr int kPerThread = kMaxRequests / kTableThreads;

// Exclusive block-wide prefix sum of one 64-bit value a thread; `total` gets the sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* wave_sum, int64_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  if (lane == 63) wave_sum[wave] = x;
  __syncthreads();
  int64_t before = 0;
  total = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 6); ++w) {
    if (w < wave) before += wave_sum[w];
    total += wave_sum[w];
  }
  __syncthreads();
  return before + x - v;
}

// The last i in [0, n) with a[i] <= v (a ascending, a[0] <= v).
__device__ __forceinline__ int last_at_most(const int32_t* a, int n, int32_t v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(kTableThreads) void page_tables(ar_page_tables_args a) {
  __shared__ int32_t q_start[kMaxRequests + 1];
  __shared__ int32_t page_at[kMaxRequests];  // pages taken by the requests before
  __shared__ uint8_t ok[kMaxRequests];
  __shared__ int64_t wave_sum[kTableThreads / 64];
  __shared__ int32_t used_pages;
  const int tid = threadIdx.x, n = a.nreq, page = a.page_size;
  const int64_t head = max(a.pool[0], 0);
  const int64_t avail = max<int64_t>(0, min(a.pool[1], a.nfree) - head);
  if (tid == 0) used_pages = 0;

  // Requests in runs of consecutive ones per thread.
  const int per = (n + kTableThreads - 1) / kTableThreads;
  int64_t tok[kPerThread], need[kPerThread], tok_sum = 0, need_sum = 0;
  bool fine[kPerThread];
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int b = tid * per + j;
    tok[j] = need[j] = 0;
    fine[j] = false;
    if (j < per && b < n) {
      const int64_t had = a.cached_len[b], add = a.new_len[b];
      const int64_t first = (had + page - 1) / page, last = (had + add + page - 1) / page;
      tok[j] = max<int64_t>(add, 0);
      fine[j] = had >= 0 && add >= 0 && last <= a.table_width && had + add <= 0x7FFFFFFF;
      need[j] = fine[j] ? last - first : 0;
    }
    tok_sum += tok[j];
    need_sum += need[j];
  }
  int64_t total, unused;
  int64_t at = block_scan(tok_sum, wave_sum, total);
  // A request whose tokens do not fit the step's buffers takes no pages.
  int64_t t = at;
  need_sum = 0;
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    t += tok[j];
    if (t > a.ntokens) fine[j] = false, need[j] = 0;
    need_sum += need[j];
  }
  int64_t pages = block_scan(need_sum, wave_sum, unused);
  int32_t used = 0;
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int b = tid * per + j;
    if (j < per && b < n) {
      const bool got = fine[j] && (need[j] == 0 || pages + need[j] <= avail);
      q_start[b] = static_cast<int32_t>(min<int64_t>(at, a.ntokens));
      page_at[b] = static_cast<int32_t>(min<int64_t>(pages, 0x7FFFFFFF));
      ok[b] = got;
      if (got && need[j] > 0) used = static_cast<int32_t>(pages + need[j]);
      if (blockIdx.x == 0) {
        const int32_t had = a.cached_len[b];
        a.kv_len[b] = got ? had + a.new_len[b] : max(had, 0);
        a.q_start[b] = q_start[b];
        a.refused[b] = !got;
      }
    }
    at += tok[j];
    pages += need[j];
  }
  if (used > 0) atomicMax(&used_pages, used);
  const int32_t end = static_cast<int32_t>(min<int64_t>(total, a.ntokens));
  if (tid == 0) q_start[n] = end;
  __syncthreads();
  const int32_t taken = used_pages;
  if (blockIdx.x == 0 && tid == 0) {
    a.q_start[n] = end;
    a.pool_out[0] = a.pool[0] + taken;
    a.pool_out[1] = a.pool[1];
  }

  const int stride = gridDim.x * kTableThreads;
  for (int i = blockIdx.x * kTableThreads + tid; i < a.ntokens; i += stride) {
    int64_t slot = -1;
    int32_t pos = -1;
    if (i < end) {
      const int b = last_at_most(q_start, n, i);
      if (ok[b]) {
        const int32_t had = a.cached_len[b];
        pos = had + i - q_start[b];
        const int32_t p = pos / page, first = static_cast<int32_t>((static_cast<int64_t>(had) + page - 1) / page);
        const int32_t id = p >= first ? a.free_pages[head + page_at[b] + p - first]
                                      : a.table[b * a.table_stride + p];
        slot = id < 0 ? -1 : static_cast<int64_t>(id) * page + pos % page;
      }
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
  }
  // New pages: entries below a request's first new page are read above, those from it on are
  // written here, so the two never meet.
  for (int i = blockIdx.x * kTableThreads + tid; i < taken; i += stride) {
    const int b = last_at_most(page_at, n, i);
    const int32_t first = static_cast<int32_t>((static_cast<int64_t>(a.cached_len[b]) + page - 1) / page);
    a.table[b * a.table_stride + first + i - page_at[b]] = a.free_pages[head + i];
  }
}

}  // namespace ard

extern "C" int ar_page_tables(const ar_page_tables_args* a, void* stream) {
  if (a == nullptr) return ar_fail(AR_EINVAL, "null arguments");
  if (a->nreq < 0 || a->ntokens < 0 || a->nfree < 0 || a->table_width < 0)
    return ar_fail(AR_EINVAL, "negative size");
  if (a->nreq > ard::kMaxRequests)
    return ar_fail(AR_ETOOBIG, "at most %d requests, got %d", ard::kMaxRequests, a->nreq);
  if (a->page_size < 1) return ar_fail(AR_EINVAL, "page_size must be positive, got %d", a->page_size);
  if (a->table_stride < a->table_width) return ar_fail(AR_EINVAL, "table_stride is below table_width");
  if (a->pool == nullptr || a->pool_out == nullptr || a->q_start == nullptr)
    return ar_fail(AR_EINVAL, "null pool or q_start");
  if (a->nreq > 0 && (a->cached_len == nullptr || a->new_len == nullptr || a->kv_len == nullptr ||
                      a->refused == nullptr || (a->table_width > 0 && a->table == nullptr)))
    return ar_fail(AR_EINVAL, "null request buffer");
  if (a->ntokens > 0 && (a->slots == nullptr || a->positions == nullptr))
    return ar_fail(AR_EINVAL, "null token buffer");
  if (a->nfree > 0 && a->free_pages == nullptr) return ar_fail(AR_EINVAL, "null free list");
  if (a->pool_out == a->pool || (a->nreq > 0 && (a->kv_len == a->cached_len || a->kv_len == a->new_len)))
    return ar_fail(AR_EINVAL, "pool_out and kv_len must not be the buffers that the call reads");
  // One workgroup up to 4096 tokens (what a decode step has), more for prompts.
  const int blocks = max(1, min(256, (a->ntokens + 4095) / 4096));
  hipLaunchKernelGGL(ard::page_tables, dim3(blocks), dim3(ard::kTableThreads), 0,
                     static_cast<hipStream_t>(stream), *a);
  AR_HIP(hipGetLastError());
  return AR_OK;
}
