// The life of a cache's pages: requests that share pages, pages copied, given back, moved together.
//
// Forks, frees and the compaction are bookkeeping on a few words a page, bound by latency: a launch, the
// lists, the tables, one atomic a page. So each workgroup repeats the short sums over all requests
// (csrc_decode/ar_decode_tables.h) and no workgroup waits for another; where something has to follow what all have done, the
// last to arrive does it. Orders are those of the lists or of the page ids, never that of arrival.
// The copy is bound by memory. Kernel times, us: a fork of 3 3.7, of 512 with 17 000 shared pages 9.0; their release 5.1 and 9.8;
// the compaction of 130 pages 2.2 + 4.6, of 33 000 6.5 + 8.8.

#include <algorithm>

#include "../../include/ar_serving.h"
#include "../csrc_decode/ar_decode_tables.h"

namespace ard {

constexpr int kMaxPages = 1 << 19;
constexpr int kFreeGrid = 256;  // workgroups of pages_free, at most

__device__ __forceinline__ uint32_t load_agent(const uint32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void store_agent(uint32_t* p, uint32_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Pages of a request, none for a negative length, at most its row's.
__device__ __forceinline__ int held_pages(int32_t len, double per_page, int width) {
  return len <= 0 ? 0 : static_cast<int>(min(pages_for(len, per_page), static_cast<uint32_t>(width)));
}

// first[b]: where request b stands first in the list, kMaxRequests where it does not.
__device__ __forceinline__ void first_places(const int32_t* list, int count, int nreq, int32_t* first) {
  for (int b = threadIdx.x; b < nreq; b += kTableThreads) first[b] = kMaxRequests;
  __syncthreads();
  for (int i = threadIdx.x; i < count; i += kTableThreads) {
    const int b = list[i];
    if (b >= 0 && b < nreq) atomicMin(&first[b], i);
  }
  __syncthreads();
}

// A workgroup takes every gridDim-th fork's row; all of them know which forks find a page.
__global__ __launch_bounds__(kTableThreads) void pages_fork(ar_pages_fork_args a, double per_page) {
  __shared__ int32_t first[kMaxRequests];
  __shared__ int32_t copied[kMaxRequests];  // the fork's tokens, -1 where it is refused
  __shared__ uint32_t taken_at[kMaxRequests];
  __shared__ uint32_t wave_sum[kMaxRequests / kTableThreads][kTableWaves];
  __shared__ uint32_t used_pages;
  const int tid = threadIdx.x;
  const int32_t pool_first = max(a.pool[0], 0);
  const int64_t head = pool_first;
  const uint32_t avail = static_cast<uint32_t>(max<int64_t>(0, min(a.pool[1], a.nfree) - head));
  if (tid == 0) used_pages = 0;
  first_places(a.dst, a.count, a.nreq, first);
  uint32_t pages = 0;
  for (int i0 = 0, round = 0; i0 < a.count; i0 += kTableThreads, ++round) {
    const int i = i0 + tid;
    int32_t len = -1;
    if (i < a.count) {
      const int src = a.src[i], dst = a.dst[i];
      if (src >= 0 && src < a.nreq && dst >= 0 && dst < a.nreq && src != dst && first[dst] == i && a.kv_len[dst] == 0) {
        len = a.kv_len[src];
        if (len > 0 && pages_for(len, per_page) > static_cast<uint32_t>(a.table_width)) len = -1;
      }
    }
    const uint32_t need = len > 0 && pages_below(len, per_page) * static_cast<uint32_t>(a.page_size) != static_cast<uint32_t>(len);
    uint32_t total;
    const uint32_t at = pages + block_scan(need, wave_sum[round], total);
    pages += total;
    if (i < a.count) {
      if (need != 0 && at >= avail) len = -1;
      copied[i] = max(len, -1);
      taken_at[i] = at;
      if (need != 0 && len >= 0) atomicMax(&used_pages, at + 1);
    }
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int b = tid; b < a.nreq; b += kTableThreads) {
      const int i = first[b];
      a.kv_len_out[b] = i < kMaxRequests && copied[i] >= 0 ? copied[i] : a.kv_len[b];
    }
    if (tid == 0) a.pool_out[0] = pool_first + static_cast<int32_t>(used_pages), a.pool_out[1] = a.pool[1];
  }
  for (int i = blockIdx.x; i < a.count; i += gridDim.x) {
    const int len = copied[i];
    const bool got = len >= 0;
    const int whole = got ? static_cast<int>(pages_below(len, per_page)) : 0;
    const bool tail = got && whole * a.page_size < len;
    const int32_t* from = got ? a.table + a.src[i] * a.table_stride : nullptr;
    int32_t* to = got ? a.table + a.dst[i] * a.table_stride : nullptr;
    for (int j = tid; j < whole; j += kTableThreads) {
      const int32_t id = from[j];
      to[j] = id;
      if (id >= 0 && id < a.num_pages) atomicAdd(&a.shares[id], 1);
    }
    if (tid == 0) {
      int32_t old = -1, own = -1;
      if (tail) {
        old = from[whole], own = a.free_pages[head + taken_at[i]];
        to[whole] = own;
      }
      a.copy_src[i] = old, a.copy_dst[i] = own;
      a.refused[i] = !got;
    }
  }
}

// Marks the pages that nobody holds any more; the last workgroup to arrive lists them.
__global__ __launch_bounds__(kTableThreads) void pages_free(ar_pages_free_args a, double per_page) {
  __shared__ int32_t first[kMaxRequests];
  __shared__ uint32_t wave_sum[2][kTableWaves];
  __shared__ uint32_t freed, before;
  const int tid = threadIdx.x, words = (a.num_pages + 31) / 32;
  uint32_t* const arrived = a.scratch + words;
  // Workgroups that have arrived, above the pages that they freed.
  constexpr uint32_t kArrived = 1u << 20;
  static_assert(kMaxPages < (1 << 20) && kFreeGrid < (1 << 12));
  if (tid == 0) freed = 0;
  first_places(a.requests, a.count, a.nreq, first);
  if (blockIdx.x == 0)
    for (int b = tid; b < a.nreq; b += kTableThreads) a.kv_len_out[b] = first[b] < kMaxRequests ? 0 : a.kv_len[b];
  for (int i = blockIdx.x; i < a.count; i += gridDim.x) {
    const int b = a.requests[i];
    if (b < 0 || b >= a.nreq || first[b] != i) continue;
    const int pages = held_pages(a.kv_len[b], per_page, a.table_width);
    const int32_t* row = a.table + b * a.table_stride;
    for (int j = tid; j < pages; j += kTableThreads) {
      const int32_t id = row[j];
      if (id < 0 || id >= a.num_pages) continue;
      if (atomicSub(&a.shares[id], 1) > 0) continue;
      const uint32_t bit = 1u << (id & 31);
      const uint32_t old = __hip_atomic_fetch_or(&a.scratch[id >> 5], bit, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if ((old & bit) == 0) atomicAdd(&freed, 1u);
    }
  }
  ar::wait_all_mem();
  __syncthreads();
  if (tid == 0) before = __hip_atomic_fetch_add(arrived, kArrived + freed, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (before / kArrived + 1 != gridDim.x) return;
  const uint32_t total = (before + freed) & (kArrived - 1);
  const int32_t pool_first = min(max(a.pool[0], 0), a.nfree);
  const int64_t start = pool_first - static_cast<int64_t>(total);
  uint32_t at = 0;
  for (int w0 = 0, round = 0; w0 < words; w0 += kTableThreads, ++round) {
    const int w = w0 + tid;
    uint32_t bits = w < words ? load_agent(a.scratch + w) : 0;
    uint32_t sum;
    int64_t to = start + at + block_scan(__popc(bits), wave_sum[round & 1], sum);
    at += sum;
    if (bits != 0) store_agent(a.scratch + w, 0);
    for (; bits != 0; bits &= bits - 1, ++to) {
      const int32_t id = w * 32 + __builtin_ctz(bits);
      a.shares[id] = 0;
      if (to >= 0) a.free_pages[to] = id;
    }
  }
  if (tid == 0) {
    a.pool_out[0] = static_cast<int32_t>(max<int64_t>(start, 0)), a.pool_out[1] = a.pool[1];
    store_agent(arrived, 0);
  }
}

__global__ __launch_bounds__(kTableThreads) void pages_mark(ar_pages_compact_args a, double per_page) {
  for (int b = blockIdx.x; b < a.nreq; b += gridDim.x) {
    const int pages = held_pages(a.kv_len[b], per_page, a.table_width);
    const int32_t* row = a.table + b * a.table_stride;
    for (int j = threadIdx.x; j < pages; j += kTableThreads) {
      const int32_t id = row[j];
      if (id >= 0 && id < a.num_pages)
        __hip_atomic_fetch_or(&a.scratch[id >> 5], 1u << (id & 31), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
}

// The pages in use as bits in LDS, with the number of them before each word.
struct Held {
  const uint32_t* bits;
  const uint32_t* before;
  // Pages held below p.
  __device__ uint32_t rank(uint32_t p) const {
    return before[p >> 5] + __popc(bits[p >> 5] & ((1u << (p & 31)) - 1));
  }
  // The k-th page below n that is not held (there is one).
  __device__ uint32_t hole(uint32_t k, uint32_t n) const {
    uint32_t lo = 0, hi = (n + 31) / 32;  // the last word with at most k before it
    while (hi - lo > 1) {
      const uint32_t mid = (lo + hi) >> 1;
      if (32 * mid - before[mid] <= k) lo = mid; else hi = mid;
    }
    uint32_t x = ~bits[lo];
    for (uint32_t left = k - (32 * lo - before[lo]); left > 0; --left) x &= x - 1;
    return 32 * lo + __builtin_ctz(x);
  }
};

__global__ __launch_bounds__(kTableThreads) void pages_compact(ar_pages_compact_args a, double per_page) {
  extern __shared__ uint32_t lds[];
  __shared__ uint32_t wave_sum[kTableWaves];
  __shared__ bool last;
  const int tid = threadIdx.x, words = (a.num_pages + 31) / 32;
  uint32_t* const bits = lds;
  uint32_t* const before = lds + words + 1;
  const int each = (words + kTableThreads) / kTableThreads;  // words of a thread; the one past the end is zero
  for (int w = tid; w <= words; w += kTableThreads) bits[w] = w < words ? load_agent(a.scratch + w) : 0;
  __syncthreads();
  uint32_t mine = 0, n;
  for (int w = tid * each; w < min((tid + 1) * each, words); ++w) mine += __popc(bits[w]);
  uint32_t at = block_scan(mine, wave_sum, n);
  for (int w = tid * each; w < min((tid + 1) * each, words + 1); ++w) before[w] = at, at += __popc(bits[w]);
  // Everyone has read the marks: the last to do so clears them.
  uint32_t* const arrived = a.scratch + words;
  if (tid == 0)
    last = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 == gridDim.x;
  __syncthreads();
  if (last)
    for (int w = tid; w <= words; w += kTableThreads) store_agent(a.scratch + w, 0);

  const Held held = {bits, before};
  const uint32_t low = held.rank(n);  // held below n: they stay
  const uint32_t moves = n - low;
  const int threads = gridDim.x * kTableThreads, me = blockIdx.x * kTableThreads + tid;
  for (int p = me; p < a.num_pages; p += threads) {
    const bool in_use = bits[p >> 5] >> (p & 31) & 1;
    a.free_pages[p] = p;
    if (p < static_cast<int>(n)) {
      if (in_use) a.shares_out[p] = a.shares[p];  // a hole's comes with the page that moves there
      continue;
    }
    a.shares_out[p] = 0;
    if (in_use) {
      const uint32_t k = held.rank(p) - low;
      const uint32_t to = held.hole(k, n);
      a.shares_out[to] = a.shares[p];
      a.move_src[k] = p, a.move_dst[k] = static_cast<int32_t>(to);
    }
  }
  for (int k = static_cast<int>(moves) + me; k < a.nmoves; k += threads) a.move_src[k] = -1, a.move_dst[k] = -1;
  if (me == 0) a.pool_out[0] = static_cast<int32_t>(n), a.pool_out[1] = a.num_pages;
  // Rows: a wave takes 64 entries of one.
  const int lane = tid & 63, chunks = (a.table_width + 63) / 64;
  const int64_t items = static_cast<int64_t>(a.nreq) * chunks;
  for (int64_t x = me >> 6; x < items; x += threads >> 6) {
    const int b = static_cast<int>(x / chunks), j = static_cast<int>(x - static_cast<int64_t>(b) * chunks) * 64 + lane;
    if (j >= a.table_width) continue;
    int32_t id = -1;
    if (j < held_pages(a.kv_len[b], per_page, a.table_width)) {
      id = a.table[b * a.table_stride + j];
      if (id >= static_cast<int>(n) && id < a.num_pages) id = held.hole(held.rank(id) - low, n);
    }
    a.table_out[b * a.out_stride + j] = id;
  }
}

constexpr int kCopyBuffers = 64, kCopyThreads = 256;
constexpr int kCopyChunk = 16384;  // bytes of a page that a workgroup takes at once
struct CopyArgs {
  uint8_t* base[kCopyBuffers];
  int64_t page_bytes[kCopyBuffers];
  int chunk_at[kCopyBuffers + 1];  // chunks of the buffers before
  uint8_t unit[kCopyBuffers];      // bytes that a thread moves at once
  const int32_t* src;
  const int32_t* dst;
  int nbuffers, count, num_pages, pairs;
};

// Copies bytes [from, from + size) of the pages of `pairs` pairs: pieces of all pairs in one row, eight of a
// thread's under way at once, written past the caches: the pages of 512 forks (0.5 GB), with fork and free, 78 us,
// 93 with plain stores, 83 with four; closing a large pool's holes (1.1 GB) 233 and 237, and 250 with a
// quarter of the pairs a workgroup.
constexpr int kCopyAhead = 8;
template <class T>
__device__ __forceinline__ void copy_pairs(uint8_t* base, int64_t page_bytes, int64_t from, int size, const int32_t* src,
                                           const int32_t* dst, int n) {
  const uint32_t pieces = size / sizeof(T), total = pieces * n;
  const float per = 1.0f / pieces;
  for (uint32_t x0 = threadIdx.x; x0 < total; x0 += kCopyAhead * kCopyThreads) {
    T v[kCopyAhead];
    int64_t to[kCopyAhead];
#pragma unroll
    for (int i = 0; i < kCopyAhead; ++i) {
      const uint32_t x = x0 + i * kCopyThreads;
      to[i] = -1;
      if (x >= total) continue;
      // x < 2^20, so the quotient is at most one off
      uint32_t pair = static_cast<uint32_t>(x * per);
      pair -= pair * pieces > x;
      pair += (pair + 1) * pieces <= x;
      const int64_t at = from + static_cast<int64_t>(x - pair * pieces) * sizeof(T);
      if (src[pair] < 0) continue;
      to[i] = dst[pair] * page_bytes + at;
      v[i] = *reinterpret_cast<const T*>(base + src[pair] * page_bytes + at);
    }
#pragma unroll
    for (int i = 0; i < kCopyAhead; ++i)
      if (to[i] >= 0) __builtin_nontemporal_store(v[i], reinterpret_cast<T*>(base + to[i]));
  }
}

__global__ __launch_bounds__(kCopyThreads) void pages_copy(CopyArgs a) {
  __shared__ int32_t src[kCopyBuffers], dst[kCopyBuffers];
  const int first = blockIdx.x * a.pairs, n = min(a.pairs, a.count - first);
  bool some = false;
  if (threadIdx.x < 64) {
    int32_t s = -1, d = -1;
    if (static_cast<int>(threadIdx.x) < n) s = a.src[first + threadIdx.x], d = a.dst[first + threadIdx.x];
    if (s < 0 || s >= a.num_pages || d < 0 || d >= a.num_pages || s == d) s = -1;
    src[threadIdx.x] = s, dst[threadIdx.x] = d;
    some = s >= 0;
  }
  if (!__syncthreads_or(some)) return;
  int b = 0, chunk = blockIdx.y;
  while (b + 1 < a.nbuffers && a.chunk_at[b + 1] <= chunk) ++b;
  chunk -= a.chunk_at[b];
  const int64_t from = static_cast<int64_t>(chunk) * kCopyChunk;
  const int size = static_cast<int>(min<int64_t>(kCopyChunk, a.page_bytes[b] - from));
  if (a.unit[b] == 16) copy_pairs<u32x4>(a.base[b], a.page_bytes[b], from, size, src, dst, n);
  else if (a.unit[b] == 4) copy_pairs<uint32_t>(a.base[b], a.page_bytes[b], from, size, src, dst, n);
  else copy_pairs<uint8_t>(a.base[b], a.page_bytes[b], from, size, src, dst, n);
}

namespace {

int check_requests(int nreq, int count, int table_width, int64_t table_stride, int page_size, int num_pages, int most) {
  if (nreq < 0 || count < 0 || table_width < 0) return ar_fail(AR_EINVAL, "negative size");
  if (nreq > kMaxRequests || count > kMaxRequests)
    return ar_fail(AR_ETOOBIG, "at most %d requests, got %d", kMaxRequests, std::max(nreq, count));
  if (page_size < 1) return ar_fail(AR_EINVAL, "page_size must be positive, got %d", page_size);
  if (table_stride < table_width) return ar_fail(AR_EINVAL, "table_stride is below table_width");
  if (num_pages < 1) return ar_fail(AR_EINVAL, "num_pages must be positive, got %d", num_pages);
  if (num_pages > most) return ar_fail(AR_ETOOBIG, "at most %d pages, got %d", most, num_pages);
  return AR_OK;
}

}  // namespace
}  // namespace ard

extern "C" {

int ar_pages_fork(const ar_pages_fork_args* a, void* stream) {
  using namespace ard;
  if (a == nullptr) return ar_fail(AR_EINVAL, "null arguments");
  if (int rc = check_requests(a->nreq, a->count, a->table_width, a->table_stride, a->page_size, a->num_pages, INT32_MAX)) return rc;
  if (a->nfree < 0) return ar_fail(AR_EINVAL, "negative size");
  if (a->pool == nullptr || a->pool_out == nullptr || a->shares == nullptr)
    return ar_fail(AR_EINVAL, "null pool or shares");
  if (a->nreq > 0 && (a->kv_len == nullptr || a->kv_len_out == nullptr || (a->table_width > 0 && a->table == nullptr)))
    return ar_fail(AR_EINVAL, "null request buffer");
  if (a->count > 0 && (a->src == nullptr || a->dst == nullptr || a->copy_src == nullptr || a->copy_dst == nullptr || a->refused == nullptr))
    return ar_fail(AR_EINVAL, "null list");
  if (a->nfree > 0 && a->free_pages == nullptr) return ar_fail(AR_EINVAL, "null free list");
  if (a->pool_out == a->pool || (a->nreq > 0 && a->kv_len_out == a->kv_len))
    return ar_fail(AR_EINVAL, "pool_out and kv_len_out must not be the buffers that the call reads");
  hipLaunchKernelGGL(pages_fork, dim3(std::max(1, std::min(a->count, 512))), dim3(kTableThreads), 0,
                     static_cast<hipStream_t>(stream), *a, 1.0 / a->page_size);
  AR_HIP(hipGetLastError());
  return AR_OK;
}

int ar_pages_free(const ar_pages_free_args* a, void* stream) {
  using namespace ard;
  if (a == nullptr) return ar_fail(AR_EINVAL, "null arguments");
  if (int rc = check_requests(a->nreq, a->count, a->table_width, a->table_stride, a->page_size, a->num_pages, kMaxPages)) return rc;
  if (a->nfree < 0) return ar_fail(AR_EINVAL, "negative size");
  if (a->pool == nullptr || a->pool_out == nullptr || a->shares == nullptr || a->scratch == nullptr)
    return ar_fail(AR_EINVAL, "null pool, shares or scratch");
  if (a->nreq > 0 && (a->kv_len == nullptr || a->kv_len_out == nullptr || (a->table_width > 0 && a->table == nullptr)))
    return ar_fail(AR_EINVAL, "null request buffer");
  if (a->count > 0 && a->requests == nullptr) return ar_fail(AR_EINVAL, "null list");
  if (a->nfree > 0 && a->free_pages == nullptr) return ar_fail(AR_EINVAL, "null free list");
  if (a->pool_out == a->pool || (a->nreq > 0 && a->kv_len_out == a->kv_len))
    return ar_fail(AR_EINVAL, "pool_out and kv_len_out must not be the buffers that the call reads");
  hipLaunchKernelGGL(pages_free, dim3(std::max(1, std::min(a->count, kFreeGrid))), dim3(kTableThreads), 0,
                     static_cast<hipStream_t>(stream), *a, 1.0 / a->page_size);
  AR_HIP(hipGetLastError());
  return AR_OK;
}

int ar_pages_compact(const ar_pages_compact_args* a, void* stream) {
  using namespace ard;
  if (a == nullptr) return ar_fail(AR_EINVAL, "null arguments");
  if (int rc = check_requests(a->nreq, 0, a->table_width, a->table_stride, a->page_size, a->num_pages, kMaxPages)) return rc;
  if (a->out_stride < a->table_width) return ar_fail(AR_EINVAL, "out_stride is below table_width");
  if (a->nfree < a->num_pages) return ar_fail(AR_EINVAL, "the free list must hold %d pages, got %d", a->num_pages, a->nfree);
  if (a->nmoves < a->num_pages / 2) return ar_fail(AR_EINVAL, "the moves must hold %d pages, got %d", a->num_pages / 2, a->nmoves);
  if (a->pool_out == nullptr || a->shares == nullptr || a->shares_out == nullptr || a->scratch == nullptr || a->free_pages == nullptr)
    return ar_fail(AR_EINVAL, "null pool, shares, free list or scratch");
  if (a->nmoves > 0 && (a->move_src == nullptr || a->move_dst == nullptr)) return ar_fail(AR_EINVAL, "null list");
  if (a->nreq > 0 && (a->kv_len == nullptr || (a->table_width > 0 && (a->table == nullptr || a->table_out == nullptr))))
    return ar_fail(AR_EINVAL, "null request buffer");
  if (a->shares_out == a->shares || (a->nreq > 0 && a->table_width > 0 && a->table_out == a->table))
    return ar_fail(AR_EINVAL, "shares_out and table_out must not be the buffers that the call reads");
  const size_t lds = ((static_cast<size_t>(a->num_pages) + 31) / 32 + 1) * 2 * sizeof(uint32_t);
  if (lds > 65536)  // more than a kernel may use unasked
    AR_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(pages_compact), hipFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(lds)));
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a->nreq > 0) {
    hipLaunchKernelGGL(pages_mark, dim3(std::min(a->nreq, 512)), dim3(kTableThreads), 0, s, *a, 1.0 / a->page_size);
    AR_HIP(hipGetLastError());
  }
  const int64_t work = a->num_pages + static_cast<int64_t>(a->nreq) * a->table_width;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(256, (work + 2 * kTableThreads - 1) / (2 * kTableThreads)));
  hipLaunchKernelGGL(pages_compact, dim3(grid), dim3(kTableThreads), lds, s, *a, 1.0 / a->page_size);
  AR_HIP(hipGetLastError());
  return AR_OK;
}

int ar_pages_copy(const ar_pages_copy_args* a, void* stream) {
  using namespace ard;
  if (a == nullptr) return ar_fail(AR_EINVAL, "null arguments");
  if (a->nbuffers < 0 || a->count < 0 || a->num_pages < 0) return ar_fail(AR_EINVAL, "negative size");
  if (a->nbuffers == 0 || a->count == 0 || a->num_pages == 0) return AR_OK;
  if (a->buffers == nullptr || a->page_bytes == nullptr || a->src == nullptr || a->dst == nullptr)
    return ar_fail(AR_EINVAL, "null list");
  for (int i = 0; i < a->nbuffers; ++i) {
    if (a->page_bytes[i] < 0) return ar_fail(AR_EINVAL, "negative size");
    if (a->buffers[i] == nullptr && a->page_bytes[i] > 0) return ar_fail(AR_EINVAL, "null buffer");
    if (a->page_bytes[i] > (int64_t(1) << 29)) return ar_fail(AR_ETOOBIG, "a page of more than 2^29 bytes");
  }
  for (int i0 = 0; i0 < a->nbuffers;) {
    // as many buffers as a launch holds, by their number and by their chunks
    CopyArgs c = {};
    int n = 0, chunks = 0;
    for (; i0 < a->nbuffers && n < kCopyBuffers; ++i0) {
      const int64_t bytes = a->page_bytes[i0];
      const int more = static_cast<int>((bytes + kCopyChunk - 1) / kCopyChunk);
      if (n > 0 && chunks + more > 65535) break;
      if (bytes == 0) continue;
      c.base[n] = static_cast<uint8_t*>(a->buffers[i0]);
      c.page_bytes[n] = bytes;
      const uintptr_t all = reinterpret_cast<uintptr_t>(c.base[n]) | static_cast<uintptr_t>(bytes);
      c.unit[n] = all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 1;
      c.chunk_at[n] = chunks, chunks += more;
      ++n;
    }
    if (n == 0) continue;
    c.chunk_at[n] = chunks;
    c.src = a->src, c.dst = a->dst, c.nbuffers = n, c.count = a->count, c.num_pages = a->num_pages;
    // Pairs of a workgroup: several where there are many, so that lists of few copies cost little.
    const int64_t all = static_cast<int64_t>(a->count) * chunks;
    c.pairs = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(64, all / 32768)));
    hipLaunchKernelGGL(pages_copy, dim3((a->count - 1) / c.pairs + 1, chunks), dim3(kCopyThreads), 0,
                       static_cast<hipStream_t>(stream), c);
    AR_HIP(hipGetLastError());
  }
  return AR_OK;
}

}  // extern "C"
