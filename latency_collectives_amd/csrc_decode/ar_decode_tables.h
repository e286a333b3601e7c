// What the kernels over block tables share: a prefix sum over a workgroup, whole pages of a length.
#pragma once

#include "ar_decode.h"

namespace ard {

constexpr int kMaxRequests = 4096;
constexpr int kTableThreads = 1024;
constexpr int kTableWaves = kTableThreads / 64;

// Exclusive block-wide prefix sum, saturating; `total` gets the sum. `wave_sum` is one call's own.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* wave_sum, uint32_t& total) {
  const uint32_t x = wave_scan(v);
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 63) wave_sum[wave] = x;
  __syncthreads();
  // lane i of every wave has the sum of wave i
  const uint32_t each = wave_scan((threadIdx.x & 63) < kTableWaves ? wave_sum[threadIdx.x & 63] : 0u);
  total = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(each), 63));
  uint32_t before = 0;
  if (wave > 0)
    before = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(each),
                                                             __builtin_amdgcn_readfirstlane(wave) - 1));
  return __builtin_elementwise_add_sat(before, x - v);
}

// n / page of any 32-bit n: n + 1/2 is at least 2^-32 of a page away from a whole number of pages,
// the product's error below 2^-51 of it.
__device__ __forceinline__ uint32_t pages_below(uint32_t n, double per_page) {
  return static_cast<uint32_t>((n + 0.5) * per_page);
}
__device__ __forceinline__ uint32_t pages_for(uint32_t n, double per_page) {
  return n == 0 ? 0 : pages_below(n - 1, per_page) + 1;
}

}  // namespace ard
