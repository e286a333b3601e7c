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

#include "ar_decode_rows.h"

namespace ard {

// Workgroups below which rows are spread over more of them. In runs of one head and of eight: one token
// of 9 heads 3.5 and 7.1 us, 1000 tokens of 16 (binary32) 5.2 and 7.0 us; 5001 tokens of 16 into the cache
// and back 21.0 and 19.1 us, 8191 of 40 67 and 33 us (inputs in the last cache).
constexpr int kFewBlocks = 512;

template <int DT, int G, int B, bool CACHE, bool PASS>
__global__ __launch_bounds__(kRowThreads) void norm_rope(RowArgs r) {
  __shared__ float stage[CACHE ? kRowThreads * 8 : 1];
  norm_rope_rows<DT, G, B, CACHE, PASS>(r, stage);
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
