// Rows of the decode path on the device: elements of either type, the sum over a row's lanes, the per-head
// norm and the rotation, rows into the 4-bit cache. ar_decode_rows.hip says how rows are shared out.
#pragma once

#include <type_traits>

#include "ar_decode.h"

namespace ard {

constexpr int kRowThreads = 256;

// Four elements of either type: as they lie in memory, as binary32, and back.
template <int DT>
struct Elem;
template <>
struct Elem<DT_F32> {
  typedef f32x4 Raw;
  __device__ static void widen(Raw v, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = v[i];
  }
  __device__ static Raw narrow(const float* x) { return Raw{x[0], x[1], x[2], x[3]}; }
  __device__ static Raw* at(const void* base, int64_t i) {
    return reinterpret_cast<Raw*>(static_cast<float*>(const_cast<void*>(base)) + i);
  }
  __device__ static float round(double y) { return static_cast<float>(y); }
};
template <>
struct Elem<DT_BF16> {
  typedef u32x2 Raw;
  __device__ static void widen(Raw v, float* x) {
    x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
  }
  __device__ static Raw narrow(const float* x) {
    return Raw{ar::bf16x2_rne(x[0], x[1]), ar::bf16x2_rne(x[2], x[3])};
  }
  __device__ static Raw* at(const void* base, int64_t i) {
    return reinterpret_cast<Raw*>(static_cast<uint16_t*>(const_cast<void*>(base)) + i);
  }
  __device__ static float round(double y) {  // by way of binary32: 2^-8 of it and 2^-24
    return bf16_lo(ar::bf16x2_rne(static_cast<float>(y), 0.0f));
  }
};
template <int DT>
__device__ __forceinline__ void load4(const void* base, int64_t i, float* x) {
  Elem<DT>::widen(*Elem<DT>::at(base, i), x);
}
// PASS: past the caches.
template <int DT, bool PASS>
__device__ __forceinline__ void store4(void* base, int64_t i, const float* x) {
  if constexpr (PASS) __builtin_nontemporal_store(Elem<DT>::narrow(x), Elem<DT>::at(base, i));
  else *Elem<DT>::at(base, i) = Elem<DT>::narrow(x);
}

// Writes eight consecutive elements x of a row, elements 8u .. 8u+7, as codes; the four lanes of a
// group of 32 share its scale. K rows are plain, V rows interleaved by four tokens.
__device__ __forceinline__ void put_row(const Cache& c, int64_t slot, int head, bool value, int d,
                                        int u, const float* x) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  most = max(most, static_cast<uint32_t>(__shfl_xor(static_cast<int>(most), 1)));
  most = max(most, static_cast<uint32_t>(__shfl_xor(static_cast<int>(most), 2)));
  // most = m 2^E with 1 <= m < 2; the smallest scale with m 2^E <= 6 scale is 2^(E-2) while
  // m <= 1.5, 2^(E-1) beyond.
  const int e = static_cast<int>(most >> 23) - 2 + ((most & 0x7FFFFFu) > 0x400000u);
  const uint32_t byte = most >= 0x7F800000u ? 255u : static_cast<uint32_t>(min(max(e, 1), kMaxScale));
  const float scale = __uint_as_float(byte << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
  if (byte == 255u) w = 0;
  const int page = 1 << c.page_shift, off = static_cast<int>(slot) & (page - 1);
  const int64_t part = ((slot >> c.page_shift) * c.heads + head) * 2 + value;
  uint8_t* data = c.data + part * (page * (d / 2));
  const int at = value ? (off >> 2) * (d * 2) + u * 16 + (off & 3) * 4 : off * (d / 2) + u * 4;
  *reinterpret_cast<uint32_t*>(data + at) = w;
  if ((u & 3) == 0) c.scales[part * (page * (d / 32)) + (u >> 2) * page + off] = static_cast<uint8_t>(byte);
}

// Between a wave's LDS stores and the loads of them by other lanes, and between those and the next
// stores. A wave's LDS accesses are done in order; this keeps them in it.
__device__ __forceinline__ void lds_turn() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Sum over the G lanes of a row, the same in each.
template <int G>
__device__ __forceinline__ double row_total(double x) {
  auto step = [&](auto ctrl) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), decltype(ctrl)::value, 0xF, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), decltype(ctrl)::value, 0xF, 0xF, false);
    x += __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
  };
  step(std::integral_constant<int, 0xB1>());   // lane ^ 1
  step(std::integral_constant<int, 0x4E>());   // lane ^ 2
  step(std::integral_constant<int, 0x141>());  // mirrored within 8
  if (G >= 16) step(std::integral_constant<int, 0x140>());  // mirrored within 16
  if (G >= 32) x += __shfl_xor(x, 16);
  return x;
}

// 1 / sqrt(a): the instruction's estimate and two Newton steps, each squaring its error.
__device__ __forceinline__ double inverse_root(double a) {
  double y = __builtin_amdgcn_rsq(a);
  if (y > 0.0) {  // not for an infinity, whose inverse root is 0, nor for NaN
    y = fma(y, fma(-0.5 * a * y, y, 0.5), y);
    y = fma(y, fma(-0.5 * a * y, y, 0.5), y);
  }
  return y;
}

// The norm (`normed`, with weights w) and the rotation (`turned`, with cosines c and sines s) of a lane's eight
// elements x, its row's G lanes together. A rotated lane has both ends of its pairs: side by side if
// interleaved, else x[j] and x[4 + j].
template <int G>
__device__ __forceinline__ void norm_rotate(const float* x, double* y, bool normed, const double* w, bool turned,
                                            const double* c, const double* s, bool interleaved, bool live,
                                            double per_dim, double eps) {
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = x[j];
  if (normed) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fma(y[j], y[j], sum);
    const double inv = inverse_root(fma(row_total<G>(live ? sum : 0.0), per_dim, eps));
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = y[j] * inv * w[j];
  }
  if (turned) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const double p = interleaved ? y[2 * j] : y[j], q = interleaved ? y[2 * j + 1] : y[4 + j];
      const double yp = p * c[j] - q * s[j], yq = q * c[j] + p * s[j];
      // what follows takes the pairs side by side or apart, as they were loaded
      if (interleaved) y[2 * j] = yp, y[2 * j + 1] = yq;
      else y[j] = yp, y[4 + j] = yq;
    }
  }
}

struct RowArgs {
  ar_qk_norm_rope_args a;
  Cache cache;
  double per_dim;  // 1 / head_dim
  int values;      // rows of v a token (kv_heads with a cache, else 0)
  int run;         // rows that a group of lanes takes
  int q_runs, k_runs;  // blocks in y: q's runs of heads, then k's, then v's
};

// G lanes a row, B rows whose loads are under way at once. CACHE: keys and values go into the cache, else keys to k_out. PASS: outputs go past
// the caches.
// stage: kRowThreads * 8 floats of LDS with CACHE. A rotated row's elements pass through it on their way to the
// cache: the rotation pairs elements half a row apart, the cache's groups are consecutive.
template <int DT, int G, int B, bool CACHE, bool PASS>
__device__ __forceinline__ void norm_rope_rows(const RowArgs& given, float* stage) {
  const RowArgs r = given;  // read at once: read where they are used, 3000 tokens of 8 heads of 96 into the cache took 6.7 us for 6.1
  const ar_qk_norm_rope_args& a = r.a;
  const int d = a.head_dim, rot = a.rot;
  const int by = blockIdx.y;
  const bool is_q = by < r.q_runs, is_v = by >= r.q_runs + r.k_runs;
  const int head0 = (is_q ? by : is_v ? by - r.q_runs - r.k_runs : by - r.q_runs) * r.run;
  const int head1 = min(head0 + r.run, is_q ? a.q_heads : is_v ? r.values : a.kv_heads);
  const int u = threadIdx.x % G;
  const int t = static_cast<int>(blockIdx.x) * (kRowThreads / G) + threadIdx.x / G;
  if (t >= a.ntokens) return;
  const int32_t pos = a.positions != nullptr ? a.positions[t] : 0;
  int64_t slot = -1;
  if (CACHE && !is_q) slot = a.slots[t];
  const void* src = is_q ? a.q : is_v ? a.v : a.k;
  const int64_t head_step = is_q ? a.q_head : is_v ? a.v_head : a.k_head;
  int64_t from = t * (is_q ? a.q_token : is_v ? a.v_token : a.k_token) + head0 * head_step;
  void* dst = is_q ? a.q_out : a.k_out;
  const int64_t to_step = is_q ? a.qo_head : a.ko_head;
  int64_t to = t * (is_q ? a.qo_token : a.ko_token) + head0 * to_step;
  const bool live = u * 8 < d;
  const bool turned = !is_v && u * 8 < rot;
  // A lane's two runs of four elements: both ends of its pairs.
  const bool halves = turned && !a.interleaved;
  const int lo = !live ? 0 : halves ? 4 * u : 8 * u, hi = !live ? 4 : halves ? rot / 2 + 4 * u : 8 * u + 4;
  typename Elem<DT>::Raw raw[B][2];
  auto load = [&](int n) {  // rows from `from` on; places past the last repeat it
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int64_t at = from + min(i, n - 1) * head_step;
      raw[i][0] = *Elem<DT>::at(src, at + lo);
      raw[i][1] = *Elem<DT>::at(src, at + hi);
    }
  };
  load(head1 - head0);
  if (pos < 0) return;
  if (CACHE && !is_q && (slot < 0 || (slot >> r.cache.page_shift) >= r.cache.num_pages)) return;
  const void* weight = is_v ? nullptr : is_q ? a.q_weight : a.k_weight;
  const bool beyond = !is_v && rot > 0 && pos >= a.rows;
  double w[8], c[4], s[4];
  if (weight != nullptr) {
    float f[8];
    load4<DT>(weight, lo, f);
    load4<DT>(weight, hi, f + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = f[i];
  }
  if (turned) {
    float f[8];
    const int64_t at = static_cast<int64_t>(beyond ? 0 : pos) * rot + 4 * u;
    load4<DT_F32>(a.cos_sin, at, f);
    load4<DT_F32>(a.cos_sin, at + rot / 2, f + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = f[i], s[i] = f[4 + i];
  }
  for (int head = head0; head < head1; head += B) {
    const int n = min(B, head1 - head);
    float x[B][8];
#pragma unroll
    for (int i = 0; i < B; ++i) Elem<DT>::widen(raw[i][0], x[i]), Elem<DT>::widen(raw[i][1], x[i] + 4);
    from += B * head_step;
    if (B > 1 && head + B < head1) load(head1 - head - B);  // the next rows, under way with these
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (i >= n) break;
      if (!is_v && (weight != nullptr || turned || beyond)) {
        double y[8];
        norm_rotate<G>(x[i], y, weight != nullptr, w, turned, c, s, a.interleaved, live, r.per_dim, a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i][j] = beyond ? __uint_as_float(0x7FC00000u) : Elem<DT>::round(y[j]);
      }
      if (CACHE && !is_q) {
        if (halves) {
          float* mine = stage + (threadIdx.x / G) * (G * 8);
#pragma unroll
          for (int j = 0; j < 4; ++j) mine[lo + j] = x[i][j], mine[hi + j] = x[i][4 + j];
          lds_turn();  // the row's lanes are one wave's
#pragma unroll
          for (int j = 0; j < 8; ++j) x[i][j] = mine[8 * u + j];
          lds_turn();  // the next row goes through the same place
        }
        if (live) put_row(r.cache, slot, head + i, is_v, d, u, x[i]);
      } else if (live) {
        store4<DT, PASS>(dst, to + i * to_step + lo, x[i]);
        store4<DT, PASS>(dst, to + i * to_step + hi, x[i] + 4);
      }
    }
    to += B * to_step;
  }
}

inline int lanes_of(int head_dim) { return head_dim <= 64 ? 8 : head_dim <= 128 ? 16 : 32; }

// ar_decode_rows.hip
int pick_run(int64_t tokens, int rows, int g);
int check_rows(const char* name, const void* p, int64_t token, int64_t head, int heads, int dtype);
int check_norm_rope(const ar_qk_norm_rope_args* a);

}  // namespace ard
