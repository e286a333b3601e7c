// The paged cache in 8 bits as the kernels see it: its codes, its scales and its handle.
#pragma once

#include "../../include/ar_serving.h"
#include "../csrc_decode/ar_decode_attn_impl.h"

namespace ard {

constexpr int kBlock = 16;  // tokens of a scale
// Scale bytes that are written: 2^-100 to 2^119. Every product of a code and one of them is a normal
// bfloat16 (or zero), so conversions are exact.
constexpr int kScale8Min = 27, kScale8Max = 246;

// Binary32 of a scale byte. What nothing wrote may be any byte: the nearer limit, so that the zeros of
// rows that do not see it meet finite values.
__device__ __forceinline__ float scale8_of(uint32_t byte) {
  return __uint_as_float(min(max(byte, static_cast<uint32_t>(kScale8Min)), static_cast<uint32_t>(kScale8Max)) << 23);
}
// Two codes (the low or the high half of w) as bfloat16, times the scale.
template <int HIGH>
__device__ __forceinline__ uint32_t codes8(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HIGH != 0));
}
// Bit 7 of every byte of w that is a NaN code.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Values beside a mask. A row's probability is 0 where it does not see a token, and 0 times an infinity or
// NaN is NaN. So in tiles that some rows see in part such values count as 0, and a product of their own
// adds them before: where `visible` (1 or 0 a place) meets one, the row's sum gets its infinity, or both
// for a NaN. This is rare and stands before the scores, where registers are left.
//
// `up` and `down`, two bfloat16 each: 1 where w's value is NaN or the infinity of that sign.
__device__ __forceinline__ void infinite_parts(uint32_t w, uint32_t& up, uint32_t& down) {
  up = down = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = w >> (16 * i) & 0xFFFFu, size = x & 0x7FFFu, one = 0x3F80u << (16 * i);
    if (size > 0x7F80u || x == 0x7F80u) up |= one;
    if (size > 0x7F80u || x == 0xFF80u) down |= one;
  }
}
__device__ __forceinline__ void add_infinite(u32x4 w, bf16x8 visible, f32x4& acc) {
  uint32_t up[4], down[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) infinite_parts(w[i], up[i], down[i]);
  const f32x4 a = mfma(operand(up[0], up[1], up[2], up[3]), visible, f32x4{0, 0, 0, 0});
  const f32x4 b = mfma(operand(down[0], down[1], down[2], down[3]), visible, f32x4{0, 0, 0, 0});
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (a[i] > 0.0f) acc[i] += INFINITY;
    if (b[i] > 0.0f) acc[i] -= INFINITY;
  }
}
// Two bfloat16 with 0 for those that are not finite.
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
  return w;
}
#define ARD_LDS __attribute__((address_space(3)))
template <class T>
__device__ __forceinline__ T lds_at(uint32_t at) {
  return *reinterpret_cast<const ARD_LDS T*>(at);
}

// Infinities and NaN that not all of a tile's rows see: 0 times them would be NaN for those that do not. Takes them
// out of `bytes` of values in LDS and tells whether there were any; a barrier before and behind is the caller's.
template <int DT, int THREADS>
__device__ __forceinline__ bool take_out(uint8_t* values, int bytes) {
  bool some = false;
  for (int x = thread_here() * 16; x < bytes; x += THREADS * 16) {
    u32x4* const p = reinterpret_cast<u32x4*>(values + x);
    const u32x4 v = *p;
    u32x4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = DT == DT_BF16 ? finite_only(v[i]) : (v[i] & 0x7F800000u) == 0x7F800000u ? 0 : v[i];
    if (y[0] != v[0] || y[1] != v[1] || y[2] != v[2] || y[3] != v[3]) some = true, *p = y;
  }
  return __any(some);
}
// The operand of 1 where sees(u, i) holds for token 4 g + i of half u.
template <class F>
__device__ __forceinline__ bf16x8 visible_of(F sees) {
  uint32_t x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = (sees(i >> 1, 2 * (i & 1)) ? 0x3F80u : 0u) | (sees(i >> 1, 2 * (i & 1) + 1) ? 0x3F800000u : 0u);
  return operand(x[0], x[1], x[2], x[3]);
}

}  // namespace ard

// The handle behind ar_kv8 is that of the 4-bit cache, with its own workspace.
struct ar_kv8 : ar_kv4 {};
