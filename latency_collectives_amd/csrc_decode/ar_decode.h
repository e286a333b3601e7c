// What the decode operators' translation units share: the cache's geometry, its codes and the
// small cross-lane helpers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/ar_decode.h"
#include "../csrc/ar_device.h"
#include "../csrc/ar_internal.h"

namespace ard {

using ar::DT_BF16;
using ar::DT_F32;
using ar::u32x2;
using ar::u32x4;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Scale bytes above this one stand for NaN: 6 * 2^(252 - 127) is the largest binary32 (and
// bfloat16) value a code can stand for, so nothing larger is ever written.
constexpr int kMaxScale = 252;

// A paged cache as a kernel sees it.
struct Cache {
  uint8_t* data;
  uint8_t* scales;
  int64_t num_pages;
  int heads;
  int page_shift;
};

// Binary32 whose exponent is the scale byte's: the scale operand of the fp4 conversions.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte > kMaxScale ? 0x7FC00000u : byte << 23);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Inclusive prefix sum over the wave's lanes, saturating.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
#define ARD_STEP(CTRL, ROWS)                  \
  x = __builtin_elementwise_add_sat(          \
      x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, ROWS, 0xF, false)));
  ARD_STEP(0x111, 0xF) ARD_STEP(0x112, 0xF) ARD_STEP(0x114, 0xF) ARD_STEP(0x118, 0xF)  // row_shr 1, 2, 4, 8
  ARD_STEP(0x142, 0xA) ARD_STEP(0x143, 0xC)  // the last lane of a row of 16, of two rows
#undef ARD_STEP
  return x;
}

}  // namespace ard

// The handle behind ar_kv4 (ar_decode_attn.hip creates it).
struct ar_kv4 {
  int heads, head_dim, page_size, page_shift;
  int device;          // where it was created, -1 without a GPU
  void* work;          // partial results, then arrival counters; NULL without a GPU
  size_t work_bytes;
};

namespace ard {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int check_handle(const ar_kv4* h) {
  return h == nullptr ? ar_fail(AR_EINVAL, "null handle") : AR_OK;
}
inline int check_dtype(int dt) {
  return dt == AR_FLOAT32 || dt == AR_BFLOAT16
             ? AR_OK
             : ar_fail(AR_ENOTSUP, "dtype must be AR_FLOAT32 or AR_BFLOAT16, got %d", dt);
}
inline int check_cache(const uint8_t* data, const uint8_t* scales, int64_t num_pages) {
  if (data == nullptr || scales == nullptr) return ar_fail(AR_EINVAL, "null cache");
  if (!aligned(data, 16) || !aligned(scales, 16))
    return ar_fail(AR_EINVAL, "the cache is not 16-byte aligned");
  if (num_pages < 1 || num_pages > (int64_t(1) << 31) - 1)
    return ar_fail(AR_EINVAL, "num_pages must be in [1, 2^31 - 1], got %lld", (long long)num_pages);
  return AR_OK;
}

}  // namespace ard
