// ar_page_tables: block tables, slots and positions of a decode step from the requests' lengths.
//
// Two prefix sums over the requests (tokens brought, pages taken) decide everything; the rest is
// one value a token or a new page. Every workgroup computes the sums of all requests for itself
// (a request's share is 8 bytes) and then fills its part of the outputs, so one launch does a step
// and no workgroup waits for another.
//
// Bound: latency. A step of a few dozen requests is two dependent loads (lengths, page ids) and
// code that runs once from a cold instruction cache, so the code is short: one copy of the scan,
// sums in 32 bits that saturate (all that they are compared with is below 2^31), a division by the
// page size as one binary64 product. In 64 bits with divisions, as first written, 32 requests of
// one token took 6.6 us and 1000 requests of up to 64 took 14.8 us; they
// take 3.3 us and 7.0 us so.

#include <algorithm>

#include "ar_decode_tables.h"

namespace ard {

// The last i in [0, n) with a[i] <= v (a ascending, a[0] <= v).
__device__ __forceinline__ int last_at_most(const uint32_t* a, int n, uint32_t v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

// Workgroups below `token_blocks` write the tokens' outputs, the others the tables' new entries.
__global__ __launch_bounds__(kTableThreads) void page_tables(ar_page_tables_args a, double per_page, int token_blocks) {
  __shared__ uint32_t q_start[kMaxRequests + 1];
  __shared__ uint32_t page_at[kMaxRequests];  // pages taken by the requests before
  __shared__ int32_t held[kMaxRequests];      // tokens of a request, -1 where it is refused
  __shared__ uint32_t wave_sum[2 * (kMaxRequests / kTableThreads)][kTableWaves];
  __shared__ uint32_t used_pages;
  const int tid = threadIdx.x, n = a.nreq;
  const uint32_t page = a.page_size, places = a.ntokens;
  const int32_t pool_first = max(a.pool[0], 0);
  const int64_t head = pool_first;
  const uint32_t avail = static_cast<uint32_t>(max<int64_t>(0, min(a.pool[1], a.nfree) - head));
  if (tid == 0) used_pages = 0;

  uint32_t tokens = 0, pages = 0;  // of the requests in the rounds before
  for (int b0 = 0, round = 0; b0 < n; b0 += kTableThreads, ++round) {
    const int b = b0 + tid;
    int32_t had = 0, add = 0;
    if (b < n) had = a.cached_len[b], add = a.new_len[b];
    const uint32_t sum = static_cast<uint32_t>(had) + static_cast<uint32_t>(add);
    const uint32_t last = pages_for(sum, per_page);
    bool fine = b < n && had >= 0 && add >= 0 && sum <= 0x7FFFFFFFu && last <= static_cast<uint32_t>(a.table_width);
    const uint32_t tok = max(add, 0);
    uint32_t total;
    const uint32_t at = __builtin_elementwise_add_sat(tokens, block_scan(tok, wave_sum[2 * round], total));
    tokens = __builtin_elementwise_add_sat(tokens, total);
    // A request whose tokens do not fit the step's buffers takes no pages.
    fine = fine && __builtin_elementwise_add_sat(at, tok) <= places;
    const uint32_t need = fine ? last - pages_for(had, per_page) : 0;
    const uint32_t taken = __builtin_elementwise_add_sat(pages, block_scan(need, wave_sum[2 * round + 1], total));
    pages = __builtin_elementwise_add_sat(pages, total);
    if (b < n) {
      const uint32_t upto = __builtin_elementwise_add_sat(taken, need);
      const bool got = fine && (need == 0 || upto <= avail);
      q_start[b] = min(at, places);
      page_at[b] = taken;
      held[b] = got ? had : -1;
      if (got && need > 0) atomicMax(&used_pages, upto);
      if (blockIdx.x == 0) {
        a.kv_len[b] = got ? had + add : max(had, 0);
        a.q_start[b] = static_cast<int32_t>(min(at, places));
        a.refused[b] = !got;
      }
    }
  }
  const uint32_t end = min(tokens, places);
  if (tid == 0) q_start[n] = end;
  __syncthreads();
  const uint32_t taken = used_pages;
  if (blockIdx.x == 0 && tid == 0) {
    a.q_start[n] = static_cast<int32_t>(end);
    a.pool_out[0] = pool_first + static_cast<int32_t>(taken);
    a.pool_out[1] = a.pool[1];
  }

  const int block = blockIdx.x;
  if (block >= token_blocks) {
    // New pages: entries below a request's first new page are only read (below), those from it on
    // only written here, so the two never meet.
    const uint32_t stride = (gridDim.x - token_blocks) * kTableThreads;
    for (uint32_t i = (block - token_blocks) * kTableThreads + tid; i < taken; i += stride) {
      const int b = last_at_most(page_at, n, i);
      a.table[b * a.table_stride + pages_for(held[b], per_page) + (i - page_at[b])] = a.free_pages[head + i];
    }
    return;
  }
  const uint32_t stride = token_blocks * kTableThreads;
  for (uint32_t i = block * kTableThreads + tid; i < places; i += stride) {
    int64_t slot = -1;
    int32_t pos = -1;
    if (i < end) {
      const int b = last_at_most(q_start, n, i);
      const int32_t had = held[b];
      if (had >= 0) {
        pos = had + static_cast<int32_t>(i - q_start[b]);
        const uint32_t p = pages_below(pos, per_page), first = pages_for(had, per_page);
        const int32_t id = p >= first ? a.free_pages[head + page_at[b] + p - first]
                                      : a.table[b * a.table_stride + p];
        slot = id < 0 ? -1 : static_cast<int64_t>(id) * page + (pos - p * page);
      }
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
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
  // A token or a new page a thread: the sums that every workgroup repeats are short against a second
  // round.
  const auto blocks = [](int64_t n) {
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(256, (n + ard::kTableThreads - 1) / ard::kTableThreads)));
  };
  const int token_blocks = blocks(a->ntokens);
  const int page_blocks = blocks(std::min<int64_t>(a->nfree, a->ntokens / a->page_size + a->nreq));
  hipLaunchKernelGGL(ard::page_tables, dim3(token_blocks + page_blocks), dim3(ard::kTableThreads), 0,
                     static_cast<hipStream_t>(stream), *a, 1.0 / a->page_size, token_blocks);
  AR_HIP(hipGetLastError());
  return AR_OK;
}
