// Rows into and out of the 8-bit paged cache, alone or with the norm and the rotation of a decode step.
//
// A block of 16 tokens of a head has one scale, so whoever writes a row has to know the other rows of its
// block: a wave takes a run (the new tokens of one block) of one head, K or V. It
// reads the run's rows (8, 16 or 32 lanes a row, eight elements a lane, as in
// csrc_decode/ar_decode_rows.h) and, where the run does not begin the block, the block's codes and scale;
// finds the largest element; puts the block together in LDS as it lies in memory; and writes what
// changed in whole 16-byte pieces. Where the scale grows, the other rows are decoded, rescaled by a power of
// two (exactly) and rounded again. Nothing is shared between waves.
//
// Bound: the launch and a few dependent loads in a decode step (slot, then rows, block and scale side by
// side): 64 tokens of 9 heads normed and rotated, one head into the cache, 4.8 us; in a prompt bytes and those loads: 8000 tokens of 8
// heads of 128 in 11 to 12 us (45 MB), the read 10 (45 MB). In and back, us, bfloat16 and binary32: those 8000 tokens 21.8 and 24.8,
// with the norm, the rotation and 8 query heads 38.7 and 41.4; 1000 single tokens of 8 heads 21.7 and 21.9, 30.9 and 30.8; 64 of one
// head 7.7 and 8.4, 7.6 and 7.8. Heads of 192 and 256 in binary32 take 38 and 44, but 114 and 134 with norm and rotation: their
// registers leave a compute unit one workgroup.

#include <algorithm>

#include "../csrc_decode/ar_decode_rows.h"
#include "ar_kv8.h"

namespace ard {

struct Put8Args {
  RowArgs r;
  int window;  // tokens that a wave looks for runs in, 1, 4 or 16
};

// Four binary32 values times `inv`, as codes. Infinities become NaN; what lies past 448 becomes that.
__device__ __forceinline__ uint32_t encode8(const float* x, float inv) {
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    y[i] = fabsf(x[i]) < INFINITY ? fminf(fmaxf(x[i] * inv, -448.0f), 448.0f) : __uint_as_float(0x7FC00000u);
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true));
}
// The same of values that are at most 448 of the scale.
__device__ __forceinline__ uint32_t scaled8(const float* x, float scale) {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  s16x2 w = {0, 0};
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[0], x[1], scale, false);
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[2], x[3], scale, true));
}
// Four codes at another scale, `ratio` of the old to the new.
__device__ __forceinline__ uint32_t rescale8(uint32_t w, float ratio) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
  int y = __builtin_amdgcn_cvt_pk_fp8_f32(lo[0] * ratio, lo[1] * ratio, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(hi[0] * ratio, hi[1] * ratio, y, true));
}
__device__ __forceinline__ uint32_t limit8(uint32_t byte) {
  return min(max(byte, static_cast<uint32_t>(kScale8Min)), static_cast<uint32_t>(kScale8Max));
}

// TURN: keys may be normed and rotated.
template <int DT, int G, bool TURN>
__device__ __forceinline__ void put8(const Put8Args& p, int head, uint8_t* image) {
  const ar_qk_norm_rope_args& a = p.r.a;
  const Cache& cache = p.r.cache;
  constexpr int AT_ONCE = 64 / G, TURNS = kBlock / AT_ONCE;  // rows, and rounds of them in a block
  constexpr int VECS = G / 8;                                // 16-byte pieces of a block a lane holds, at most
  const int d = a.head_dim, rot = a.rot, shift = cache.page_shift, page = 1 << shift;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool is_v = (wave & 1) != 0;
  const int first = (static_cast<int>(blockIdx.x) * (kRowThreads / 128) + (wave >> 1)) * p.window;
  if (first >= a.ntokens) return;

  // Lane i has the slot of token first - 15 + i, -1 where nothing is written. The tokens of a run keep step
  // with their slots, so the rest of a token's run is among the 15 tokens before it and the 15 after it.
  constexpr int LOOK = kBlock - 1;
  int64_t slot = -1;
  int place = -1;  // its position, below 0 for a token that is skipped
  {
    const int t = first - LOOK + lane;
    if (t >= 0 && t < a.ntokens) {
      slot = a.slots[t];
      place = a.positions != nullptr ? a.positions[t] : 0;
    }
    if (slot < 0 || (slot >> shift) >= cache.num_pages || place < 0) slot = -1;
  }
  const int u = lane % G, sub = lane / G;
  const bool live = u * 8 < d;
  const bool turned = TURN && !is_v && u * 8 < rot;
  const bool halves = turned && !a.interleaved;
  const int lo = !live ? 0 : halves ? 4 * u : 8 * u, hi = !live ? 4 : halves ? rot / 2 + 4 * u : 8 * u + 4;
  const void* src = is_v ? a.v : a.k;
  const int64_t token_step = is_v ? a.v_token : a.k_token;
  const int64_t head_at = head * (is_v ? a.v_head : a.k_head);
  const bool normed = TURN && !is_v && a.k_weight != nullptr;
  double w[8];
  if (normed) {
    float f[8];
    load4<DT>(a.k_weight, lo, f);
    load4<DT>(a.k_weight, hi, f + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = f[i];
  }

  uint64_t left = __ballot(slot >= 0 && lane >= LOOK && lane < LOOK + p.window);
  while (left != 0) {
    const int leader = __builtin_ctzll(left);
    const uint64_t at = static_cast<uint64_t>(static_cast<uint32_t>(lane_value(static_cast<uint32_t>(slot >> 32), leader))) << 32 |
                        static_cast<uint32_t>(lane_value(static_cast<uint32_t>(slot), leader));
    // The tokens of its run: those of the block that keep step with it.
    const int64_t mine = static_cast<int64_t>(at);
    const uint64_t run = __ballot((slot >> 4) == (mine >> 4) && slot - mine == lane - leader);
    left &= ~run;
    if (__builtin_ctzll(run) < leader) continue;  // an earlier token leads it
    const int t0 = first - LOOK + leader;
    const int in_page = static_cast<int>(at) & (page - 1), o = in_page & (kBlock - 1);
    const int64_t owner = static_cast<int64_t>(at >> shift) * cache.heads + head;
    uint8_t* block = cache.data + (owner * 2 + is_v) * (static_cast<int64_t>(page) * d) + (in_page - o) * d;
    uint8_t* scale = cache.scales + owner * (2 * (page / kBlock)) + in_page / kBlock * 2 + is_v;
    const bool fresh = o == 0;
    const uint64_t members = run >> leader;  // counted from the first; skipped ones may lie between
    const int n = 64 - __builtin_clzll(members);

    typename Elem<DT>::Raw raw[TURNS][2];
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
      if (i * AT_ONCE >= n) break;
      const int64_t from = (t0 + min(i * AT_ONCE + sub, n - 1)) * token_step + head_at;
      raw[i][0] = *Elem<DT>::at(src, from + lo);
      raw[i][1] = *Elem<DT>::at(src, from + hi);
    }
    u32x4 old[VECS];
    uint32_t old_byte = 0;
    if (!fresh) {
      old_byte = *scale;
#pragma unroll
      for (int i = 0; i < VECS; ++i) old[i] = reinterpret_cast<const u32x4*>(block)[min(lane + 64 * i, d - 1)];
    }

    float x[TURNS][8];  // only with TURN: else as loaded, and widened twice
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
      if (i * AT_ONCE >= n) break;
      const int row = i * AT_ONCE + sub;
      float now[8];
      Elem<DT>::widen(raw[i][0], now), Elem<DT>::widen(raw[i][1], now + 4);
      if (TURN && (normed || (!is_v && rot > 0))) {
        // a skipped token's position is below 0: its row is computed and not used
        const int pos = max(__shfl(place, leader + min(row, n - 1)), 0);
        const bool beyond = rot > 0 && pos >= a.rows;
        double c[4], s[4], y[8];
        if (turned) {
          float f[8];
          const int64_t from = static_cast<int64_t>(beyond ? 0 : pos) * rot + 4 * u;
          load4<DT_F32>(a.cos_sin, from, f);
          load4<DT_F32>(a.cos_sin, from + rot / 2, f + 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) c[j] = f[j], s[j] = f[4 + j];
        }
        norm_rotate<G>(now, y, normed, w, turned, c, s, a.interleaved, live, p.r.per_dim, a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) now[j] = beyond ? __uint_as_float(0x7FC00000u) : Elem<DT>::round(y[j]);
      }
      if (live && (members >> row & 1) != 0)
#pragma unroll
        for (int j = 0; j < 8; ++j) most = max(most, __float_as_uint(now[j]) & 0x7FFFFFFFu);
      if constexpr (TURN) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i][j] = now[j];
      } else {
        asm("" : "+v"(raw[i][0]), "+v"(raw[i][1]));
      }
    }
    most = wave_max(most);
    auto row_of = [&](int i) {
      if constexpr (!TURN) Elem<DT>::widen(raw[i][0], x[i]), Elem<DT>::widen(raw[i][1], x[i] + 4);
      return x[i];
    };
    const bool wild = most >= 0x7F800000u;
    if (wild) {  // infinities and NaN have no part in the scale
      most = 0;
#pragma unroll
      for (int i = 0; i < TURNS; ++i) {
        if (i * AT_ONCE >= n) break;
        const float* y = row_of(i);
        if (live && (members >> (i * AT_ONCE + sub) & 1) != 0)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t size = __float_as_uint(y[j]) & 0x7FFFFFFFu;
            if (size < 0x7F800000u) most = max(most, size);
          }
      }
      most = wave_max(most);
    }
    // most = m 2^E with 1 <= m < 2, and 448 = 1.75 * 2^8.
    const int need = static_cast<int>(most >> 23) - 8 + ((most & 0x7FFFFFu) > 0x600000u);
    uint32_t byte = static_cast<uint32_t>(min(max(need, kScale8Min), kScale8Max));
    const uint32_t had = limit8(uniform(static_cast<int>(old_byte)));
    if (!fresh) byte = max(byte, had);
    const bool grown = !fresh && byte > had;
    // Else every value is at most 448 of the scale, and two conversions give a word.
    const bool careful = wild || need > kScale8Max;
    const float unit = __uint_as_float(byte << 23), inv = __uint_as_float((254u - byte) << 23);
    // 448 * 2^-30 is nothing beside the smallest code, 2^-9.
    const float ratio = byte - had < 30u ? __uint_as_float((127u - (byte - had)) << 23) : 0.0f;

    // The block as it lies in memory.
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int x16 = lane + 64 * i;
      if (x16 >= d) continue;
      u32x4 v = {0, 0, 0, 0};
      if (!fresh) {
        v = old[i];
        if (grown)
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = rescale8(v[j], ratio);
      }
      reinterpret_cast<u32x4*>(image)[x16] = v;
    }
    lds_turn();
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
      if (i * AT_ONCE >= n) break;
      const int row = i * AT_ONCE + sub;
      if (!live || (members >> row & 1) == 0) continue;
      const float* y = row_of(i);
      uint32_t c0, c1;
      if (careful) c0 = encode8(y, inv), c1 = encode8(y + 4, inv);
      else c0 = scaled8(y, unit), c1 = scaled8(y + 4, unit);
      const int token = o + row;
      if (!is_v) {
        *reinterpret_cast<uint32_t*>(image + token * d + lo) = c0;
        *reinterpret_cast<uint32_t*>(image + token * d + hi) = c1;
      } else {
        uint8_t* to = image + (token >> 2) * (4 * d) + u * 32 + (token & 3);
#pragma unroll
        for (int j = 0; j < 4; ++j) to[4 * j] = static_cast<uint8_t>(c0 >> (8 * j)), to[16 + 4 * j] = static_cast<uint8_t>(c1 >> (8 * j));
      }
    }
    lds_turn();
    int from = 0, upto = d;  // 16-byte pieces that changed
    if (!fresh && !grown) {
      // d / 16 pieces a key's row, d / 4 four tokens' values
      from = is_v ? (o >> 2) * (d / 4) : o * (d / 16);
      upto = is_v ? ((o + n + 3) >> 2) * (d / 4) : (o + n) * (d / 16);
    }
    for (int i = from + lane; i < upto; i += 64)
      reinterpret_cast<u32x4*>(block)[i] = reinterpret_cast<const u32x4*>(image)[i];
    if (lane == 0 && (fresh || byte != old_byte)) *scale = static_cast<uint8_t>(byte);
    lds_turn();  // the next run goes through the same place
  }
}

// Blocks of y: q's runs of heads as in norm_rope (none without a norm), then the cache's heads.
template <int DT, int G, int B>
__global__ __launch_bounds__(kRowThreads) void kv8_put(Put8Args p) {
  __shared__ u32x4 image[kRowThreads / 64][G * 8];  // a block of each wave, 16 rows of up to 8 G bytes
  const int by = blockIdx.y;
  if (by < p.r.q_runs) {
    norm_rope_rows<DT, G, B, false, false>(p.r, nullptr);
    return;
  }
  put8<DT, G, true>(p, by - p.r.q_runs, reinterpret_cast<uint8_t*>(image[threadIdx.x >> 6]));
}

template <int DT, int G>
__global__ __launch_bounds__(kRowThreads) void kv8_append(Put8Args p) {
  __shared__ u32x4 image[kRowThreads / 64][G * 8];
  put8<DT, G, false>(p, blockIdx.y, reinterpret_cast<uint8_t*>(image[threadIdx.x >> 6]));
}

struct Read8Args {
  ar_kv8_rows_args a;
  Cache cache;
  int head_dim;
};

template <int DT, int G>
__global__ __launch_bounds__(kRowThreads) void kv8_read(Read8Args r) {
  const ar_kv8_rows_args& a = r.a;
  const int u = threadIdx.x % G, d = r.head_dim;
  const int t = static_cast<int>(blockIdx.x) * (kRowThreads / G) + threadIdx.x / G;
  if (t >= a.ntokens || u * 8 >= d) return;
  const bool value = static_cast<int>(blockIdx.y) >= r.cache.heads;
  const int head = value ? blockIdx.y - r.cache.heads : blockIdx.y;
  const int64_t slot = a.slots[t];
  float x[8] = {};
  if (slot >= 0 && (slot >> r.cache.page_shift) < r.cache.num_pages) {
    const int page = 1 << r.cache.page_shift, off = static_cast<int>(slot) & (page - 1);
    const int64_t owner = (slot >> r.cache.page_shift) * r.cache.heads + head;
    const uint8_t* data = r.cache.data + (owner * 2 + value) * (static_cast<int64_t>(page) * d);
    const float scale = scale8_of(r.cache.scales[owner * (2 * (page / kBlock)) + off / kBlock * 2 + value]);
    uint32_t c[2];
    if (!value) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(data + off * d + 8 * u);
      c[0] = v.x, c[1] = v.y;
    } else {
      const u32x4* p = reinterpret_cast<const u32x4*>(data + (off >> 2) * (4 * d) + u * 32);
      const int by = 8 * (off & 3);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const u32x4 v = p[i];
        c[i] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i] |= (v[j] >> by & 0xFFu) << (8 * j);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t y0 = codes8<0>(c[i], scale), y1 = codes8<1>(c[i], scale);
      x[4 * i] = bf16_lo(y0), x[4 * i + 1] = bf16_hi(y0), x[4 * i + 2] = bf16_lo(y1), x[4 * i + 3] = bf16_hi(y1);
    }
  }
  void* dst = value ? a.v : a.k;
  const int64_t to = (value ? t * a.v_token + head * a.v_head : t * a.k_token + head * a.k_head) + 8 * u;
  store4<DT, false>(dst, to, x);
  store4<DT, false>(dst, to + 4, x + 4);
}

namespace {

// Tokens that a wave looks for runs in. The host does not know the runs: tokens of a decode step are one each, a prompt's 16.
// With a wave for a token all are under way at once, most of a prompt's waves find that another has theirs; with 16 a wave
// takes a decode step's runs one after the other. Into a cache of 8 heads of 128 and back, us with 1, 4 and 16: 256
// single tokens (4096 waves) 10.5, 12.9, 24.2; 512 15.2, 17.0, 29.1 (normed and rotated 20.5, 20.5, 37.1); 1000 34.2, 31.6,
// 45.4 normed and rotated; a prompt of 600 9.7, 9.6, 8.8, of 1000 19.9, 15.3, 12.1 normed and rotated, of 2000 15.3, 11.4,
// 11.0, of 4000 (64 000) 24.5, 17.9, 16.1.
int window_of(int64_t waves) { return waves < 8192 ? 1 : waves < 65536 ? 4 : 16; }

int launch_put(RowArgs& r, hipStream_t stream) {
  const int g = lanes_of(r.a.head_dim), heads = r.a.kv_heads;
  if (r.a.ntokens == 0) return AR_OK;
  r.per_dim = 1.0 / r.a.head_dim;
  r.run = r.a.q_heads > 0 ? pick_run(r.a.ntokens, r.a.q_heads, g) : 1;
  r.q_runs = (r.a.q_heads + r.run - 1) / r.run;
  Put8Args p{r, window_of(static_cast<int64_t>(r.a.ntokens) * heads * 2)};
  if (r.q_runs + heads > 65535) return ar_fail(AR_ETOOBIG, "too many heads");
  const auto blocks = [](int64_t n, int64_t each) { return static_cast<unsigned>((n + each - 1) / each); };
  unsigned in_x = blocks(r.a.ntokens, p.window * (kRowThreads / 128));
  if (r.q_runs > 0) in_x = std::max(in_x, blocks(r.a.ntokens, kRowThreads / g));
  const dim3 grid(in_x, r.q_runs + heads), block(kRowThreads);
  void (*fn)(Put8Args);
  const bool plain = r.q_runs == 0 && r.a.k_weight == nullptr && r.a.rot == 0;
#define ARD_PICK(DT, G) fn = plain ? kv8_append<DT, G> : r.run == 1 ? kv8_put<DT, G, 1> : kv8_put<DT, G, 4>
  if (r.a.dtype == AR_BFLOAT16) {
    if (g == 8) ARD_PICK(DT_BF16, 8); else if (g == 16) ARD_PICK(DT_BF16, 16); else ARD_PICK(DT_BF16, 32);
  } else {
    if (g == 8) ARD_PICK(DT_F32, 8); else if (g == 16) ARD_PICK(DT_F32, 16); else ARD_PICK(DT_F32, 32);
  }
#undef ARD_PICK
  hipLaunchKernelGGL(fn, grid, block, 0, stream, p);
  AR_HIP(hipGetLastError());
  return AR_OK;
}

Cache cache8_of(const ar_kv8* h, uint8_t* data, uint8_t* scales, int64_t num_pages) {
  return Cache{data, scales, num_pages, h->heads, h->page_shift};
}

int check_rows8(const ar_kv8* h, const ar_kv8_rows_args* a) {
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

}  // namespace
}  // namespace ard

extern "C" {

int ar_kv8_append(ar_kv8* h, const ar_kv8_rows_args* a, void* stream) {
  if (int rc = ard::check_rows8(h, a)) return rc;
  ard::RowArgs r{};
  r.a.k = a->k, r.a.v = a->v, r.a.slots = a->slots;
  r.a.k_token = a->k_token, r.a.k_head = a->k_head, r.a.v_token = a->v_token, r.a.v_head = a->v_head;
  r.a.dtype = a->dtype, r.a.ntokens = a->ntokens, r.a.kv_heads = h->heads, r.a.head_dim = h->head_dim;
  r.cache = ard::cache8_of(h, a->data, a->scales, a->num_pages);
  return ard::launch_put(r, static_cast<hipStream_t>(stream));
}

int ar_kv8_norm_rope_append(ar_kv8* h, const ar_qk_norm_rope_args* a, void* stream) {
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
  ard::RowArgs r{*a, ard::cache8_of(h, a->data, a->scales, a->num_pages), 0.0, 0, 0, 0, 0};
  return ard::launch_put(r, static_cast<hipStream_t>(stream));
}

int ar_kv8_read(ar_kv8* h, const ar_kv8_rows_args* a, void* stream) {
  if (int rc = ard::check_rows8(h, a)) return rc;
  if (a->ntokens == 0) return AR_OK;
  const int g = ard::lanes_of(h->head_dim), each = ard::kRowThreads / g;
  const dim3 grid((a->ntokens - 1) / each + 1, 2 * h->heads), block(ard::kRowThreads);
  const ard::Read8Args r{*a, ard::cache8_of(h, a->data, a->scales, a->num_pages), h->head_dim};
  hipStream_t s = static_cast<hipStream_t>(stream);
#define ARD_LAUNCH(DT, G) hipLaunchKernelGGL((ard::kv8_read<ard::DT, G>), grid, block, 0, s, r)
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
