// Row operators of the decode path: per-head RMS norm and position rotation of q and k, rows into
// the 4-bit paged cache and rows out of it.
//
// A row (one head of one token, 64..256 elements) belongs to 8, 16 or 32 neighbouring lanes, eight
// elements a lane, so everything a row needs (its sum of squares, the largest element of each 32)
// is a few cross-lane steps and each byte of HBM moves once. A group of lanes takes `run`
// neighbouring heads of one token, four rows' loads under way at once; the token's cosines and the
// weights are read and widened once for them.
//
// Arithmetic of the norm and the rotation is 64-bit: gfx950's binary64 rate is that of unpacked
// binary32, the kernel is bound by bytes (or by its launch), and what is rounded to bfloat16 and
// then to 4 bits hardly depends on the order of the sum of squares.
//
// Measured, 8191 tokens of 32 + 8 heads of 128 in bfloat16 (172 MB): 38.7 us, 4.4 TB/s; one row a group
// with a 64-bit division for its place and a library square root and reciprocal was bound by its
// instructions (56 us).

#include <type_traits>

#include "ar_decode.h"

namespace ard {

constexpr int kRowThreads = 256;
// Workgroups below which rows are spread over more of them. In runs of one head and of eight: one token
// of 9 heads 3.5 and 7.1 us, 1000 tokens of 16 (binary32) 5.2 and 7.0 us; 5001 tokens of 16 into the cache
// and back 21.0 and 19.1 us, 8191 of 40 67 and 33 us (inputs in the last cache).
constexpr int kFewBlocks = 512;

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
template <int DT, int G, int B, bool CACHE, bool PASS>
__global__ __launch_bounds__(kRowThreads) void norm_rope(RowArgs r) {
  const ar_qk_norm_rope_args& a = r.a;
  // A rotated row's elements pass through LDS on their way to the cache: the rotation pairs
  // elements half a row apart, the cache's groups are consecutive.
  __shared__ float stage[CACHE ? kRowThreads * 8 : 1];
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
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[i][j];
        if (weight != nullptr) {
          double sum = 0.0;
#pragma unroll
          for (int j = 0; j < 8; ++j) sum = fma(y[j], y[j], sum);
          const double inv = inverse_root(fma(row_total<G>(live ? sum : 0.0), r.per_dim, a.eps));
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = y[j] * inv * w[j];
        }
        if (turned) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const double p = a.interleaved ? y[2 * j] : y[j], q = a.interleaved ? y[2 * j + 1] : y[4 + j];
            const double yp = p * c[j] - q * s[j], yq = q * c[j] + p * s[j];
            // what follows takes the pairs side by side or apart, as they were loaded
            if (a.interleaved) y[2 * j] = yp, y[2 * j + 1] = yq;
            else y[j] = yp, y[4 + j] = yq;
          }
        }
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

struct ReadArgs {
  ar_kv4_rows_args a;
  Cache cache;
  int head_dim;
};

template <int DT, int G>
__global__ __launch_bounds__(kRowThreads) void read_rows(ReadArgs r) {
  const ar_kv4_rows_args& a = r.a;
  const int u = threadIdx.x % G, d = r.head_dim;
  const int t = static_cast<int>(blockIdx.x) * (kRowThreads / G) + threadIdx.x / G;
  if (t >= a.ntokens || u * 8 >= d) return;
  const bool value = blockIdx.y >= r.cache.heads;
  const int head = value ? blockIdx.y - r.cache.heads : blockIdx.y;
  const int64_t slot = a.slots[t];
  float x[8] = {};
  if (slot >= 0 && (slot >> r.cache.page_shift) < r.cache.num_pages) {
    const int page = 1 << r.cache.page_shift, off = static_cast<int>(slot) & (page - 1);
    const int64_t part = ((slot >> r.cache.page_shift) * r.cache.heads + head) * 2 + value;
    const int at = value ? (off >> 2) * (d * 2) + u * 16 + (off & 3) * 4 : off * (d / 2) + u * 4;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(r.cache.data + part * (page * (d / 2)) + at);
    const float scale = scale_of(r.cache.scales[part * (page * (d / 32)) + (u >> 2) * page + off]);
    const uint32_t p[4] = {
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3))};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(p[i]), x[2 * i + 1] = bf16_hi(p[i]);
  }
  void* dst = value ? a.v : a.k;
  const int64_t to = (value ? t * a.v_token + head * a.v_head : t * a.k_token + head * a.k_head) + 8 * u;
  store4<DT, false>(dst, to, x);
  store4<DT, false>(dst, to + 4, x + 4);
}

inline int lanes_of(int head_dim) { return head_dim <= 64 ? 8 : head_dim <= 128 ? 16 : 32; }

// Heads that a group of lanes takes, of `heads`: eight, half as many while the launch would not give
// every compute unit a few workgroups (then one row a group: latency counts).
int pick_run(int64_t tokens, int rows, int g) {
  const int64_t blocks = (tokens * g + kRowThreads - 1) / kRowThreads;
  int run = 8;
  while (run > 1 && blocks * ((rows + run - 1) / run) < kFewBlocks) run /= 2;
  return run;
}

template <bool CACHE>
int launch_norm_rope(RowArgs& r, hipStream_t stream) {
  const int g = lanes_of(r.a.head_dim);
  const int rows = r.a.q_heads + r.a.kv_heads + r.values;
  if (r.a.ntokens == 0 || rows == 0) return AR_OK;
  r.per_dim = 1.0 / r.a.head_dim;
  r.run = pick_run(r.a.ntokens, rows, g);
  // More than the XCDs' L2 hold (32 MiB) is not read from there again. Through the caches and past them,
  // 40 heads of 128 in bfloat16, 16, 30, 36 and 80 MiB of outputs: 13.3 and 12.0, 16.7 and 14.6, 20.8
  // and 18.1, 42.5 and 38.0 us alone; with an elementwise call that reads q after them 18.7 and 18.1,
  // 27.4 and 27.7, 33.0 and 34.7, 63.2 and 66.0 us. So the threshold is the L2's size, and what a
  // call gains alone below it, or its reader above, is within 15 % and 5 %.
  // Only where every store is of neighbouring lanes' neighbouring elements: halves of lines that
  // go past the L2 one by one took 29 us for 8000 tokens of 17 interleaved heads of 64 in binary32, 18 us through it.
  const bool pass = !CACHE && !r.a.interleaved && r.a.rot == r.a.head_dim &&
                    static_cast<int64_t>(r.a.ntokens) * (r.a.q_heads + r.a.kv_heads) * r.a.head_dim *
                            (r.a.dtype == AR_BFLOAT16 ? 2 : 4) > (int64_t(32) << 20);
  const auto runs = [&](int heads) { return (heads + r.run - 1) / r.run; };
  r.q_runs = runs(r.a.q_heads), r.k_runs = runs(r.a.kv_heads);
  const int in_y = r.q_runs + r.k_runs + runs(r.values);
  if (in_y > 65535) return ar_fail(AR_ETOOBIG, "too many heads");
  const int each = kRowThreads / g;
  const dim3 grid((r.a.ntokens + each - 1) / each, in_y), block(kRowThreads);
  void (*fn)(RowArgs);
  // One row a group has its own, shorter code: one token's 9 heads 2.7 us, 3.4 us with room for four.
#define ARD_PICK(DT, G)                                  \
  fn = r.run == 1 ? norm_rope<DT, G, 1, CACHE, false>    \
       : pass     ? norm_rope<DT, G, 4, CACHE, !CACHE>   \
                  : norm_rope<DT, G, 4, CACHE, false>
  if (r.a.dtype == AR_BFLOAT16) {
    if (g == 8) ARD_PICK(DT_BF16, 8); else if (g == 16) ARD_PICK(DT_BF16, 16); else ARD_PICK(DT_BF16, 32);
  } else {
    if (g == 8) ARD_PICK(DT_F32, 8); else if (g == 16) ARD_PICK(DT_F32, 16); else ARD_PICK(DT_F32, 32);
  }
#undef ARD_PICK
  hipLaunchKernelGGL(fn, grid, block, 0, stream, r);
  AR_HIP(hipGetLastError());
  return AR_OK;
}

// Base address and strides of a [tokens][heads][head_dim] tensor in units of four elements.
int check_rows(const char* name, const void* p, int64_t token, int64_t head, int heads, int dtype) {
  if (heads == 0) return AR_OK;
  if (p == nullptr) return ar_fail(AR_EINVAL, "null %s", name);
  if (!aligned(p, dtype == AR_BFLOAT16 ? 8 : 16) || token % 4 != 0 || head % 4 != 0)
    return ar_fail(AR_EINVAL, "%s: address and strides must be multiples of 4 elements", name);
  if (token < 0 || head < 0) return ar_fail(AR_EINVAL, "%s: negative stride", name);
  return AR_OK;
}

int check_norm_rope(const ar_qk_norm_rope_args* a) {
  if (a == nullptr) return ar_fail(AR_EINVAL, "null arguments");
  if (int rc = check_dtype(a->dtype)) return rc;
  if (a->ntokens < 0 || a->q_heads < 0 || a->kv_heads < 0) return ar_fail(AR_EINVAL, "negative size");
  if (a->q_heads > 65536 || a->kv_heads > 65536) return ar_fail(AR_ETOOBIG, "too many heads");
  if (a->head_dim < 8 || a->head_dim > 256 || a->head_dim % 8 != 0)
    return ar_fail(AR_EINVAL, "head_dim must be a multiple of 8 in [8, 256], got %d", a->head_dim);
  if (a->rot < 0 || a->rot > a->head_dim || a->rot % 8 != 0)
    return ar_fail(AR_EINVAL, "rot must be a multiple of 8 in [0, head_dim], got %d", a->rot);
  if (!(a->eps >= 0)) return ar_fail(AR_EINVAL, "eps must not be negative");
  if (a->ntokens == 0) return AR_OK;
  if (a->rot > 0 && (a->positions == nullptr || a->cos_sin == nullptr || a->rows < 1))
    return ar_fail(AR_EINVAL, "a rotation needs positions and cos_sin");
  if (a->rot > 0 && !aligned(a->cos_sin, 16)) return ar_fail(AR_EINVAL, "cos_sin is not 16-byte aligned");
  const uintptr_t w = a->dtype == AR_BFLOAT16 ? 8 : 16;
  if (!aligned(a->q_weight, w) || !aligned(a->k_weight, w))
    return ar_fail(AR_EINVAL, "a weight's address must be a multiple of 4 elements");
  if (int rc = check_rows("q", a->q, a->q_token, a->q_head, a->q_heads, a->dtype)) return rc;
  if (int rc = check_rows("k", a->k, a->k_token, a->k_head, a->kv_heads, a->dtype)) return rc;
  if (int rc = check_rows("q_out", a->q_out, a->qo_token, a->qo_head, a->q_heads, a->dtype)) return rc;
  if (a->q_heads > 0 && a->q == a->q_out && (a->q_token != a->qo_token || a->q_head != a->qo_head))
    return ar_fail(AR_EINVAL, "q in place needs equal strides");
  return AR_OK;
}

Cache cache_of(const ar_kv4* h, uint8_t* data, uint8_t* scales, int64_t num_pages) {
  return Cache{data, scales, num_pages, h->heads, h->page_shift};
}

int check_kv_rows(const ar_kv4* h, const ar_kv4_rows_args* a) {
  if (int rc = check_handle(h)) return rc;
  if (a == nullptr) return ar_fail(AR_EINVAL, "null arguments");
  if (int rc = check_dtype(a->dtype)) return rc;
  if (a->ntokens < 0) return ar_fail(AR_EINVAL, "negative size");
  if (int rc = check_cache(a->data, a->scales, a->num_pages)) return rc;
  if (a->ntokens == 0) return AR_OK;
  if (a->slots == nullptr) return ar_fail(AR_EINVAL, "null slots");
  if (int rc = check_rows("k", a->k, a->k_token, a->k_head, h->heads, a->dtype)) return rc;
  return check_rows("v", a->v, a->v_token, a->v_head, h->heads, a->dtype);
}

}  // namespace ard

extern "C" {

int ar_qk_norm_rope(const ar_qk_norm_rope_args* a, void* stream) {
  if (int rc = ard::check_norm_rope(a)) return rc;
  if (a->ntokens > 0) {
    if (int rc = ard::check_rows("k_out", a->k_out, a->ko_token, a->ko_head, a->kv_heads, a->dtype)) return rc;
    if (a->kv_heads > 0 && a->k == a->k_out && (a->k_token != a->ko_token || a->k_head != a->ko_head))
      return ar_fail(AR_EINVAL, "k in place needs equal strides");
  }
  ard::RowArgs r{*a, {}, 0.0, 0, 0, 0, 0};
  return ard::launch_norm_rope<false>(r, static_cast<hipStream_t>(stream));
}

int ar_kv4_norm_rope_append(ar_kv4* h, const ar_qk_norm_rope_args* a, void* stream) {
  if (int rc = ard::check_handle(h)) return rc;
  if (int rc = ard::check_norm_rope(a)) return rc;
  if (a->kv_heads != h->heads || a->head_dim != h->head_dim)
    return ar_fail(AR_EINVAL, "the handle is for %d kv heads of %d, got %d of %d", h->heads, h->head_dim,
                   a->kv_heads, a->head_dim);
  if (int rc = ard::check_cache(a->data, a->scales, a->num_pages)) return rc;
  if (a->ntokens > 0) {
    if (a->slots == nullptr) return ar_fail(AR_EINVAL, "null slots");
    if (int rc = ard::check_rows("v", a->v, a->v_token, a->v_head, a->kv_heads, a->dtype)) return rc;
  }
  ard::RowArgs r{*a, ard::cache_of(h, a->data, a->scales, a->num_pages), 0.0, a->kv_heads, 0, 0, 0};
  return ard::launch_norm_rope<true>(r, static_cast<hipStream_t>(stream));
}

int ar_kv4_append(ar_kv4* h, const ar_kv4_rows_args* a, void* stream) {
  if (int rc = ard::check_kv_rows(h, a)) return rc;
  ard::RowArgs r{};
  r.a.k = a->k, r.a.v = a->v, r.a.slots = a->slots;
  r.a.k_token = a->k_token, r.a.k_head = a->k_head, r.a.v_token = a->v_token, r.a.v_head = a->v_head;
  r.a.dtype = a->dtype, r.a.ntokens = a->ntokens, r.a.kv_heads = h->heads, r.a.head_dim = h->head_dim;
  r.cache = ard::cache_of(h, a->data, a->scales, a->num_pages);
  r.values = h->heads;
  return ard::launch_norm_rope<true>(r, static_cast<hipStream_t>(stream));
}

int ar_kv4_read(ar_kv4* h, const ar_kv4_rows_args* a, void* stream) {
  if (int rc = ard::check_kv_rows(h, a)) return rc;
  const int g = ard::lanes_of(h->head_dim);
  if (a->ntokens == 0) return AR_OK;
  const int each = ard::kRowThreads / g;
  const dim3 grid((a->ntokens + each - 1) / each, 2 * h->heads), block(ard::kRowThreads);
  const ard::ReadArgs r{*a, ard::cache_of(h, a->data, a->scales, a->num_pages), h->head_dim};
  hipStream_t s = static_cast<hipStream_t>(stream);
#define ARD_LAUNCH(DT, G) hipLaunchKernelGGL((ard::read_rows<ard::DT, G>), grid, block, 0, s, r)
  if (a->dtype == AR_BFLOAT16) {
    if (g == 8) ARD_LAUNCH(DT_BF16, 8); else if (g == 16) ARD_LAUNCH(DT_BF16, 16); else ARD_LAUNCH(DT_BF16, 32);
  } else {
    if (g == 8) ARD_LAUNCH(DT_F32, 8); else if (g == 16) ARD_LAUNCH(DT_F32, 16); else ARD_LAUNCH(DT_F32, 32);
  }
#undef ARD_LAUNCH
  AR_HIP(hipGetLastError());
  return AR_OK;
}

}  // extern "C"
