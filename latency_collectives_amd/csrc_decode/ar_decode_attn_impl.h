// Attention over the 4-bit paged cache (gfx950).
//
// Mathematics. One pass over the keys and values with a running reference m and sum l per row:
// s = scale q.k in base-2 units, p = 2^(s - m), l += p, o += p v; where a row's maximum passes m by
// more than 8, l and o are scaled by 2^(m - m') first (p then stays below 2^8, far from any
// limit). Parts of a row are joined by the same rule. m starts from a finite value: a masked score
// (minus infinity) less it is minus infinity without a test, and a NaN score, which a maximum
// passes over, still reaches l. So l is 0 only where a row sees nothing.
//
// Shape. The products run transposed, so that nothing is moved between lanes in the loop:
//   S^T [32 tokens x 16 rows]  = K  [tokens x D]  Q^T      two 16x16x32 tiles
//   O^T [D x 16 rows]         += V^T [D x tokens] P^T
// A lane (c = lane % 16, g = lane / 16) of the first product holds row c's scores of tokens
// 4g .. 4g+3 of both 16-token halves, which is exactly its operand of the second. Keys: a lane
// reads a quarter of token c's row, its operand of every step along D. Values: a lane reads eight
// elements of four tokens at once (the cache's interleaved layout) and pairs tokens with one byte
// permute per pair. Codes become bfloat16 with one conversion per two elements, the scale applied
// by the conversion, exactly; no LDS is used before the join. Probabilities of bfloat16 calls
// are rounded to bfloat16 (by 2^-8 at most, under a result that is rounded by as much): results of 8
// requests of up to 131072 tokens are off by 0.0022 of their norm, by 0.0017 with their own rounding
// alone. A second part a probability took 129 us for them against 125, and 37 % more for prompt chunks.
//
// Work. A job is a tile of query rows (16 * NQ: tokens x heads of the group) of one request and kv
// head; its tokens are 32-token units. All jobs' units in one row are cut into equal runs, one run a
// workgroup, whose four waves take every fourth unit. A run may end one job, hold whole ones and
// begin another, so every workgroup reads the same number of bytes whatever the requests' lengths
// are (64 requests of up to 8192 tokens, 8 kv heads of 128, 285 MB: 85 us with one part of a job a
// workgroup, which left a second, half-empty round of workgroups; 63 us so). A job
// of several workgroups leaves partial sums in the workspace and the last one to arrive joins them
// in the order of the tokens, so the result does not depend on who came last. Nothing waits for
// another workgroup.
#pragma once

#include "ar_decode_attn.h"

namespace ard {

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ bf16x8 operand(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
  const u32x4 v = {w0, w1, w2, w3};
  return __builtin_bit_cast(bf16x8, v);
}
template <int BYTE>
__device__ __forceinline__ uint32_t codes(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, BYTE));
}
// Low (high) halves of a and b side by side.
__device__ __forceinline__ uint32_t pair_lo(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t pair_hi(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// Over the four lanes that hold one row: lane ^ 16, lane ^ 32.
__device__ __forceinline__ float row_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float row_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}
__device__ __forceinline__ int row_or(int x) {
  x |= __shfl_xor(x, 16);
  return x | __shfl_xor(x, 32);
}
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// A running maximum that no score has reached yet: the lowest finite value.
constexpr float kLowest = -3.4028235e38f;

// x as a sum of PARTS bfloat16 values (three hold all 24 bits). An infinity or NaN stays in the
// first part alone.
template <int PARTS>
__device__ __forceinline__ void split(const float* x, bf16x8* out) {
  uint32_t w[PARTS][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      uint32_t v;
      if (p + 1 < PARTS) {
        // truncated, so that no finite value becomes infinite
        v = pair_hi(__float_as_uint(a), __float_as_uint(b));
        const float ra = a - bf16_lo(v), rb = b - bf16_hi(v);
        a = fabsf(a) < INFINITY ? ra : 0.0f;
        b = fabsf(b) < INFINITY ? rb : 0.0f;
      } else {
        v = ar::bf16x2_rne(a, b);
      }
      w[p][i] = v;
    }
  }
#pragma unroll
  for (int p = 0; p < PARTS; ++p) out[p] = operand(w[p][0], w[p][1], w[p][2], w[p][3]);
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
#define ARD_STEP(CTRL, ROWS) \
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, ROWS, 0xF, false)));
  ARD_STEP(0x111, 0xF) ARD_STEP(0x112, 0xF) ARD_STEP(0x114, 0xF) ARD_STEP(0x118, 0xF)
  ARD_STEP(0x142, 0xA) ARD_STEP(0x143, 0xC)
#undef ARD_STEP
  return __builtin_amdgcn_readlane(static_cast<int>(x), 63);
}
__device__ __forceinline__ int lane_value(uint32_t x, int lane) {
  return __builtin_amdgcn_readlane(static_cast<int>(x), lane);
}

// A request as the split sees it: tiles of rows, and their units: the tokens that a tile may see and,
// after them, what starting and ending a job costs in units.
struct Cost {
  int q0, m, kv;
  int tiles, span;
};

template <int R>
__device__ __forceinline__ Cost cost_of(const AttnArgs& args, int b) {
  const ar_kv4_attention_args& a = args.a;
  Cost c = {0, 0, 0, 0, 1};
  if (b < a.nreq) {
    const int at = a.q_start[b], to = a.q_start[b + 1];
    c.kv = max(a.kv_len[b], 0);
    c.q0 = min(max(at, 0), a.ntokens);
    c.m = max(min(to, a.ntokens) - c.q0, 0);
    c.tiles = static_cast<int>((static_cast<uint32_t>(c.m) * static_cast<uint32_t>(args.group) + R - 1) / R);
    const uint32_t seen = min(static_cast<uint32_t>(c.kv), args.most_seen);
    c.span = static_cast<int>((seen + args.unit - 1) >> args.unit_shift) + args.job_units;
  }
  return c;
}

// Where a workgroup is in its run: a job and the units of it.
struct Run {
  int request, tile, head;
  int at;    // the job's first unit of this run
  int left;  // units of the run from there on
  int per;   // units of a run
};

// The run of workgroup `w`; false where there is none. Every wave computes it alone (lanes are
// requests), with no barrier. This code runs once, from a cold instruction cache, before anything
// else: it is kept short (32-bit sums; the host picks units large enough for them).
template <int R>
__device__ __forceinline__ bool find_run(const AttnArgs& args, int w, Run& run, Cost& mine) {
  const int lane = threadIdx.x & 63, heads = args.cache.heads;
  uint32_t total = 0, longest = 0;
  Cost c;
  uint32_t upto;
  for (int b = (args.a.nreq - 1) & ~63; b >= 0; b -= 64) {  // ends with the first requests at hand
    c = cost_of<R>(args, b + lane);
    upto = wave_scan(static_cast<uint32_t>(c.tiles * heads) * static_cast<uint32_t>(c.span));
    total = __builtin_elementwise_add_sat(total, static_cast<uint32_t>(lane_value(upto, 63)));
    longest = max(longest, wave_max(c.tiles > 0 ? c.span : 0));
  }
  // Only request starts that overlap reach this: nothing is done.
  if (total > 0x7FFFFFFFu) return false;
  // A unit for each wave at least, and no more parts of a job than units of a part: reading a part
  // back costs about what a unit does where few jobs leave the device idle.
  const int least = max((total + args.runs - 1) / args.runs,
                        static_cast<uint32_t>(uniform(static_cast<int>(sqrtf(static_cast<float>(longest))))));
  run.per = max(kAttnWaves, (least + kAttnWaves - 1) & ~(kAttnWaves - 1));
  if (static_cast<uint64_t>(w) * run.per >= total) return false;
  uint32_t from = w * run.per;
  run.left = min(run.per, static_cast<int>(total - from));
  int b = 0;
  while (__ballot(upto > from) == 0) {
    from -= lane_value(upto, 63);
    b += 64;
    if (b >= args.a.nreq) return false;  // only if lengths change under the call
    c = cost_of<R>(args, b + lane);
    upto = wave_scan(static_cast<uint32_t>(c.tiles * heads) * static_cast<uint32_t>(c.span));
  }
  const int who = __builtin_ctzll(__ballot(upto > from));
  run.request = b + who;
  mine.q0 = lane_value(c.q0, who), mine.m = lane_value(c.m, who), mine.kv = lane_value(c.kv, who);
  mine.tiles = lane_value(c.tiles, who), mine.span = lane_value(c.span, who);
  from += static_cast<uint32_t>(mine.tiles * heads) * static_cast<uint32_t>(mine.span) - lane_value(upto, who);
  // Jobs in the order of the heads, a head's tiles side by side: they share its keys.
  const uint32_t job = from / static_cast<uint32_t>(mine.span);
  run.at = uniform(from - job * mine.span);
  run.head = uniform(job), run.tile = 0;
  if (mine.tiles > 1) {
    run.head = uniform(job / static_cast<uint32_t>(mine.tiles));
    run.tile = uniform(job - run.head * mine.tiles);
  }
  return true;
}

// The next job of the run.
template <int R>
__device__ __forceinline__ void next_job(const AttnArgs& args, Run& run, Cost& mine) {
  run.at = 0;
  if (++run.tile < mine.tiles) return;
  run.tile = 0;
  if (++run.head < args.cache.heads) return;
  run.head = 0;
  do {
    if (++run.request >= args.a.nreq) {  // only if lengths change under the call
      run.left = 0;
      return;
    }
    mine = cost_of<R>(args, run.request);
    mine.tiles = uniform(mine.tiles);
  } while (mine.tiles == 0);
  mine.q0 = uniform(mine.q0), mine.m = uniform(mine.m), mine.kv = uniform(mine.kv), mine.span = uniform(mine.span);
}

// The first position that a row at `pos` sees with a window. Positions below 0 see nothing and count
// as -1: less a window of nearly 2^31 they would wrap to a positive start, which the tile's other
// rows would miss their tokens by.
__device__ __forceinline__ int window_start(int pos, int window) { return max(pos, -1) - window + 1; }

// Memory that a computed address is known to lie in: a load of unknown place counts as one from
// LDS too, and every wait for LDS would wait for it.
#define ARD_GLOBAL __attribute__((address_space(1)))
typedef const ARD_GLOBAL uint8_t* global_bytes;
template <class T>
__device__ __forceinline__ T load_at(global_bytes base, uint32_t off) {
  asm("" : "+v"(off));  // stays a 32-bit offset beside a scalar base
  return *reinterpret_cast<const ARD_GLOBAL T*>(base + off);
}
// The address that lane `l` holds.
__device__ __forceinline__ global_bytes lane_address(uint64_t x, int l) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(x), l);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(x >> 32), l);
  return reinterpret_cast<global_bytes>(static_cast<uint64_t>(hi) << 32 | lo);
}

// Any byte above kMaxScale (252) in a word of scale bytes.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x03030303u) & w & 0x80808080u;
}

// N consecutive dwords with the widest loads that their alignment allows (4 N bytes, N a divisor or
// multiple of the width).
template <int N>
__device__ __forceinline__ void load_dwords(global_bytes p, uint32_t off, uint32_t* out) {
  constexpr int W = N % 4 == 0 ? 4 : N % 2 == 0 ? 2 : 1;
  typedef uint32_t vec __attribute__((ext_vector_type(W)));
#pragma unroll
  for (int i = 0; i < N; i += W) {
    const vec v = load_at<vec>(p, off + 4 * i);
#pragma unroll
    for (int j = 0; j < W; ++j) out[i + j] = v[j];
  }
}

template <int D>
struct Tile32 {  // a lane's share of 32 tokens, as loaded
  static constexpr int kDw = D / 32;               // dwords of a quarter of a K row
  static constexpr int kKs = kDw == 2 || kDw == 4 ? 1 : 2;  // 32-groups they lie in
  static constexpr int kSets = (D / 8 + 15) / 16;  // chunks of eight elements / 16 lanes
  uint32_t k[2][kDw];
  uint32_t ks[2][kKs];
  u32x4 v[2][kSets];
  uint32_t vs[2][kSets];
};

// Eight elements of a row of `out` from its sums, and its logarithm.
template <int DT>
__device__ __forceinline__ void finish_row(const ar_kv4_attention_args& a, int64_t token, int head, int seg,
                                           f32x4 o0, f32x4 o1, float top, float rl) {
  const float inv = rl == 0.0f ? 0.0f : 1.0f / rl;
  o0 *= inv, o1 *= inv;
  const int64_t to = token * a.o_token + head * a.o_head + seg * 8;
  if (DT == DT_BF16) {
    const u32x4 w = {ar::bf16x2_rne(o0[0], o0[1]), ar::bf16x2_rne(o0[2], o0[3]),
                     ar::bf16x2_rne(o1[0], o1[1]), ar::bf16x2_rne(o1[2], o1[3])};
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + to) = w;
  } else {
    *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + to) = o0;
    *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + to + 4) = o1;
  }
  if (seg == 0 && a.lse != nullptr)
    a.lse[token * a.q_heads + head] = rl == 0.0f ? -INFINITY : (top + log2f(rl)) * 0.6931471805599453f;
}

// Counts this workgroup's part of a job as done; true in the last of `parts`. Write-through stores
// are done before the arrival is counted.
__device__ __forceinline__ bool arrive(uint32_t* arrived, int parts, int* last) {
  ar::wait_all_mem();
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t before = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *last = before + 1 == static_cast<uint32_t>(parts);
    if (*last) __hip_atomic_store(arrived, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return *last;
}

// Joins a job's parts, in the order of the tokens. A thread reads eight elements of a row from
// every part, or from every `groups`-th where threads are left over; N parts are under way at once.
template <int D, int R, int N, class F>
__device__ __forceinline__ void join_parts(ar::rsrc_t part, uint32_t stats_at, int first_wg, int parts, int rows,
                                           float* lds, F finish) {
  constexpr int NC = D / 8;
  const int tid = threadIdx.x, items = rows * NC;
  int groups = 1;
  while (groups * 2 * items <= kAttnThreads && groups * N < parts) groups *= 2;
  for (int x0 = 0; x0 < items * groups; x0 += kAttnThreads) {
    const int x = x0 + tid, mine = x / items, y = x - mine * items;
    const int r = y / NC, seg = y - r * NC;
    float top = -INFINITY, rl = 0.0f;
    f32x4 o0 = {0, 0, 0, 0}, o1 = {0, 0, 0, 0};
    for (int p0 = mine; p0 < parts && mine < groups; p0 += N * groups) {
      u32x2 st[N];
      u32x4 v0[N], v1[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int p = min(p0 + k * groups, parts - 1);
        // slot of part p > 0 is 2 * (first_wg + p), of part 0 one more than 2 * first_wg
        const uint32_t at = static_cast<uint32_t>((2 * (first_wg + p) + (p == 0)) * R + r);
        st[k] = ar::ld8<ar::kCoh>(part, stats_at + at * 8);
        v0[k] = ar::ld16<ar::kCoh>(part, (at * D + seg * 8) * 4);
        v1[k] = ar::ld16<ar::kCoh>(part, (at * D + seg * 8 + 4) * 4);
      }
      float to = top;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (p0 + k * groups >= parts) st[k].x = 0xFF800000u;  // -infinity
        to = fmaxf(to, __uint_as_float(st[k].x));
      }
      const float f0 = exp2_fast(top - to);
      o0 *= f0, o1 *= f0, rl *= f0;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float f = exp2_fast(__uint_as_float(st[k].x) - to);
        rl += __uint_as_float(st[k].y) * f;
        o0 += __builtin_bit_cast(f32x4, v0[k]) * f, o1 += __builtin_bit_cast(f32x4, v1[k]) * f;
      }
      top = to;
    }
    if (groups > 1) {  // one round of the outer loop: the groups' sums meet in LDS
      if (x < items * groups) {
        float* p = lds + x * 12;
        *reinterpret_cast<f32x4*>(p) = o0;
        *reinterpret_cast<f32x4*>(p + 4) = o1;
        p[8] = top, p[9] = rl;
      }
      __syncthreads();
      if (x < items)
        for (int k = 1; k < groups; ++k) {
          const float* p = lds + (k * items + x) * 12;
          const float to = fmaxf(top, p[8]);
          const float f0 = exp2_fast(top - to), f1 = exp2_fast(p[8] - to);
          o0 = o0 * f0 + *reinterpret_cast<const f32x4*>(p) * f1;
          o1 = o1 * f0 + *reinterpret_cast<const f32x4*>(p + 4) * f1;
          rl = rl * f0 + p[9] * f1, top = to;
        }
    }
    if (x < items) finish(r, seg, o0, o1, top, rl);
  }
}

// The same for many rows and at most N parts: a thread has N parts of I segments under way at once.
template <int D, int R, int N, int I, class F>
__device__ __forceinline__ void join_few(ar::rsrc_t part, uint32_t stats_at, int first_wg, int parts, int rows,
                                         F finish) {
  constexpr int NC = D / 8;
  const int items = rows * NC;
  for (int x0 = threadIdx.x; x0 < items; x0 += I * kAttnThreads) {
    u32x2 st[I][N];
    u32x4 v0[I][N], v1[I][N];
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int x = min(x0 + i * kAttnThreads, items - 1), r = x / NC, seg = x - r * NC;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int p = min(k, parts - 1);
        const uint32_t at = static_cast<uint32_t>((2 * (first_wg + p) + (p == 0)) * R + r);
        st[i][k] = ar::ld8<ar::kCoh>(part, stats_at + at * 8);
        v0[i][k] = ar::ld16<ar::kCoh>(part, (at * D + seg * 8) * 4);
        v1[i][k] = ar::ld16<ar::kCoh>(part, (at * D + seg * 8 + 4) * 4);
      }
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int x = x0 + i * kAttnThreads, r = x / NC, seg = x - r * NC;
      float top = -INFINITY, rl = 0.0f;
      f32x4 o0 = {0, 0, 0, 0}, o1 = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (k < parts) top = fmaxf(top, __uint_as_float(st[i][k].x));
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (k >= parts) continue;
        const float f = exp2_fast(__uint_as_float(st[i][k].x) - top);
        rl += __uint_as_float(st[i][k].y) * f;
        o0 += __builtin_bit_cast(f32x4, v0[i][k]) * f, o1 += __builtin_bit_cast(f32x4, v1[i][k]) * f;
      }
      if (x < items) finish(r, seg, o0, o1, top, rl);
    }
  }
}

template <int DT, int D, int NQ, int OCC>
__global__ __launch_bounds__(kAttnThreads, OCC) void kv4_attention(AttnArgs args) {
  constexpr int R = 16 * NQ;
  constexpr int PARTS = DT == DT_BF16 ? 1 : 3;
  constexpr int NC = D / 8;
  typedef Tile32<D> Tile;
  constexpr int kDw = Tile::kDw, kKs = Tile::kKs, kSets = Tile::kSets;
  // Registers for two tiles of keys are not left: the next ones are loaded behind the scores.
  constexpr bool kLate = kSets == 2 && NQ == 2;
  constexpr int kPitch = D + 4;  // LDS row: 16 rows' 16-byte accesses fall into different banks
  __shared__ float join[kAttnWaves * 16 * kPitch];
  __shared__ float stat_m[kAttnWaves][R], stat_l[kAttnWaves][R];
  __shared__ int last;

  const ar_kv4_attention_args& a = args.a;
  const int w = blockIdx.x;
  Run run;
  Cost me;
  if (!find_run<R>(args, w, run, me)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int group = args.group, shift = args.cache.page_shift;
  // Per-lane offsets within a page's K and V.
  const int page = 1 << shift;
  const int k_bytes = page * (D / 2), s_bytes = page * (D / 32);
  const int num_pages = static_cast<int>(args.cache.num_pages);
  const int k_group = (g * kDw) >> 2;  // 32-group of a lane's first K dword
  const uint32_t k_off = c * (D / 2) + g * (D / 8);
  uint32_t v_off[kSets], vs_off[kSets];
#pragma unroll
  for (int e = 0; e < kSets; ++e) {
    const int chunk = min(e * 16 + c, NC - 1);  // lanes beyond the row repeat its last chunk
    v_off[e] = k_bytes + g * (D * 2) + chunk * 16;
    vs_off[e] = s_bytes + (chunk >> 2) * page + g * 4;
  }

  for (;;) {
    // Rows of this tile and what each sees.
    const int rows = me.m * group;
    const int row0 = run.tile * R;
    int i0 = 0;
    if (run.tile > 0) i0 = uniform(static_cast<uint32_t>(row0) / static_cast<uint32_t>(group));
    const int rem0 = row0 - i0 * group;
    // token and head in the group of row row0 + r: rem0 + r is below 2^17, exact in binary32
    auto token_of = [&](int r) { return static_cast<int>((rem0 + r + 0.5f) * args.per_group); };
    const int i1 = i0 + uniform(token_of(min(R, rows - row0) - 1));
    const int kv_end = min(me.kv, args.room);
    const int first_pos = me.kv - me.m;  // position of the request's first new token
    const int end = min(max(first_pos + i1 + 1, 0), kv_end);
    int begin = 0;
    if (a.window > 0) begin = max(window_start(first_pos + i0, a.window), 0) & ~31;
    const int ntiles = end > begin ? (end - begin + 31) >> 5 : 0;
    if (ntiles == 0) begin = 0;  // the window may begin anywhere past the table: no place is computed from there
    const int nunits = (ntiles + (1 << args.tile_shift) - 1) >> args.tile_shift;
    const int taken = min(run.left, me.span - run.at);  // units of the run in this job
    const int t_first = run.at << args.tile_shift;
    const int t_last = min((run.at + taken) << args.tile_shift, ntiles);
    run.left -= taken;
    // Parts of the job: part 0 is the workgroup that holds its first unit, slot 2 * (that) + 1; the
    // others hold nothing before it in their runs, slot 2 * (theirs).
    int before = 0, first_units = taken;  // parts before this one, units of part 0
    if (run.at > 0) {
      before = uniform(static_cast<uint32_t>(run.at + run.per - 1) / static_cast<uint32_t>(run.per));
      first_units = run.at - (before - 1) * run.per;
    }
    const int first_wg = w - before;
    int parts = 1;
    if (nunits > first_units)
      parts = 1 + uniform(static_cast<uint32_t>(nunits - first_units + run.per - 1) / static_cast<uint32_t>(run.per));
    if (run.at == 0 || t_first < ntiles) {
      const uint8_t* data = args.cache.data + static_cast<int64_t>(run.head) * 2 * k_bytes;
      const uint8_t* scales = args.cache.scales + static_cast<int64_t>(run.head) * 2 * s_bytes;
      const int32_t* table = a.table + run.request * a.table_stride;

      // Where the keys of this wave's next 32 tiles and their scales start: lane 2 k + u has the u-th
      // half of the k-th, a valid place where there is nothing to see. One page id a tile would make
      // the wave wait for its keys and values with it.
      auto pages = [&](int tile) {
        const int mine = tile + (lane >> 1) * kAttnWaves, t = begin + mine * 32 + (lane & 1) * 16;
        return mine < t_last && t < end ? table[t >> shift] : -1;
      };
      uint64_t k_at, s_at, seen;
      auto settle = [&](int p) {
        const bool some = p >= 0 && p < num_pages;
        const int64_t at = some ? p : 0;
        const int off = (begin + (t_first + wave) * 32 + (lane & 1) * 16 + (lane >> 1) * (kAttnWaves * 32)) & (page - 1);
        k_at = reinterpret_cast<uint64_t>(data) + at * args.page_bytes + off * (D / 2);
        s_at = reinterpret_cast<uint64_t>(scales) + at * args.page_scales + off;
        seen = __ballot(some);
      };
      int ids = pages(t_first + wave);  // under way with the queries

      int hi[NQ], lo[NQ];
      bf16x8 q[NQ][PARTS][kDw];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const int row = row0 + n * 16 + c;
        const bool real = row < rows;  // others repeat the last row, with nothing to see
        const int r = min(n * 16 + c, rows - 1 - row0), i = i0 + token_of(r);
        const int pos = first_pos + i;
        hi[n] = real ? min(pos + 1, kv_end) : 0;
        lo[n] = a.window > 0 ? window_start(pos, a.window) : 0;
        const int64_t at = static_cast<int64_t>(me.q0 + i) * a.q_token +
                           static_cast<int64_t>(run.head * group + row0 + r - i * group) * a.q_head + g * (D / 4);
#pragma unroll
        for (int s = 0; s < kDw; ++s) {
          if (DT == DT_BF16) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.q) + at + s * 8);
            q[n][0][s] = __builtin_bit_cast(bf16x8, w);
          } else {
            float x[8];
            const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(a.q) + at + s * 8);
            const f32x4 v0 = p[0], v1 = p[1];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = v0[j], x[4 + j] = v1[j];
            bf16x8 w[PARTS];
            split<PARTS>(x, w);
#pragma unroll
            for (int p = 0; p < PARTS; ++p) q[n][p][s] = w[p];
          }
        }
      }
      // Tiles from here on need masks: the first row's end, the last row's window.
      const int whole_end = min(first_pos + i0 + 1, kv_end);
      const int whole_begin = a.window > 0 ? window_start(first_pos + i1, a.window) : 0;

      f32x4 acc[NQ][kSets][8];
      float m[NQ], l[NQ];
      int nan_groups[NQ];  // groups of 32 elements in which a visible value is NaN
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        m[n] = kLowest, l[n] = 0.0f, nan_groups[n] = 0;
#pragma unroll
        for (int e = 0; e < kSets; ++e)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[n][e][j] = f32x4{0, 0, 0, 0};
      }

      auto load_keys = [&](int k, Tile& x) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const global_bytes kd = lane_address(k_at, 2 * k + u), sd = lane_address(s_at, 2 * k + u);
          load_dwords<kDw>(kd, k_off, x.k[u]);
#pragma unroll
          for (int s = 0; s < kKs; ++s)
            x.ks[u][s] = load_at<uint8_t>(sd, min(k_group + s, D / 32 - 1) * page + c);
        }
      };
      auto load_values = [&](int k, Tile& x) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const global_bytes kd = lane_address(k_at, 2 * k + u), sd = lane_address(s_at, 2 * k + u);
#pragma unroll
          for (int e = 0; e < kSets; ++e) {
            x.v[u][e] = load_at<u32x4>(kd, v_off[e]);
            x.vs[u][e] = load_at<uint32_t>(sd, vs_off[e]);
          }
        }
      };

      // The first round only loads: one copy of this code.
      Tile now, next;
      int tile = t_first + wave - kAttnWaves, turn = 0;
      int both = 0, both_next;  // the halves that have a page
      for (; tile < t_last; tile += kAttnWaves) {
        if ((turn & 31) == 0) {
          settle(ids);
          ids = pages(tile + 33 * kAttnWaves);
        }
        both_next = static_cast<int>(seen >> (2 * (turn & 31))) & 3;
        const int k_next = turn++ & 31;
        if (!kLate) load_keys(k_next, next);
        load_values(k_next, next);
        f32x4 s[NQ][2];
        const int t0 = begin + tile * 32;
        // Scores.
        if (tile >= t_first) {
#pragma unroll
          for (int n = 0; n < NQ; ++n) s[n][0] = s[n][1] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float sc[kKs];
#pragma unroll
            for (int i = 0; i < kKs; ++i) sc[i] = scale_of(now.ks[u][i]);
#pragma unroll
            for (int i = 0; i < kDw; ++i) {
              float x = sc[0];
              if (kKs > 1) x = ((g * kDw + i) >> 2) == k_group ? sc[0] : sc[kKs - 1];
              const uint32_t w = now.k[u][i];
              const bf16x8 kk = operand(codes<0>(w, x), codes<1>(w, x), codes<2>(w, x), codes<3>(w, x));
#pragma unroll
              for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int p = 0; p < PARTS; ++p) s[n][u] = mfma(kk, q[n][p][i], s[n][u]);
            }
          }
        }
        if (kLate) load_keys(k_next, now);
        if (tile >= t_first) {
          const bool partial = t0 + 32 > whole_end || t0 < whole_begin || both != 3;
#pragma unroll
          for (int n = 0; n < NQ; ++n) s[n][0] *= args.scale_log2, s[n][1] *= args.scale_log2;
          if (partial) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int t = t0 + u * 16 + g * 4 + i;
                  if (t >= hi[n] || t < lo[n] || (both >> u & 1) == 0) s[n][u][i] = -INFINITY;
                }
          }

          // Values that are NaN (or bytes that were never written) must not meet the zeros of rows that
          // do not see them: such groups are read as finite and the rows that do see them noted.
          uint32_t odd = 0;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < kSets; ++e) odd |= nan_bytes(now.vs[u][e]);
          if (__any(odd != 0)) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int e = 0; e < kSets; ++e) {
                uint32_t bad = nan_bytes(now.vs[u][e]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {  // the groups of this set, held by lanes c = 4k
                  const int group32 = e * 4 + k;
                  if (group32 >= D / 32) break;
                  const uint32_t theirs = __shfl(static_cast<int>(bad), g * 16 + 4 * k);
#pragma unroll
                  for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                      const int t = t0 + u * 16 + g * 4 + i;
                      if ((theirs >> (8 * i + 7) & 1) && t < hi[n] && t >= lo[n] && (both >> u & 1) != 0)
                        nan_groups[n] |= 1 << group32;
                    }
                }
                bad |= bad >> 1, bad |= bad >> 2, bad |= bad >> 4;
                now.vs[u][e] &= ~bad;  // 2^-127 or so: finite
              }
          }

          // Probabilities.
          bf16x8 pr[NQ][PARTS];
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = s[n][i >> 2][i & 3];
            float top = x[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top = fmaxf(top, x[i]);
            if (__any(top > m[n] + 8.0f)) {
              const float to = fmaxf(m[n], row_max(top));
              const float f = exp2_fast(m[n] - to);
              m[n] = to;
              l[n] *= f;
#pragma unroll
              for (int e = 0; e < kSets; ++e)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[n][e][j] *= f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              x[i] = exp2_fast(x[i] - m[n]);
              l[n] += x[i];
            }
            split<PARTS>(x, pr[n]);
          }

          // Values.
#pragma unroll
          for (int e = 0; e < kSets; ++e) {
            float sc[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              sc[i] = __uint_as_float((now.vs[i >> 2][e] >> (8 * (i & 3)) & 0xFFu) << 23);
#define ARD_PAIR(B)                                                                              \
  {                                                                                              \
    uint32_t w[8];                                                                               \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) w[i] = codes<B>(now.v[i >> 2][e][i & 3], sc[i]); \
    const bf16x8 v0 = operand(pair_lo(w[0], w[1]), pair_lo(w[2], w[3]), pair_lo(w[4], w[5]),     \
                              pair_lo(w[6], w[7]));                                              \
    const bf16x8 v1 = operand(pair_hi(w[0], w[1]), pair_hi(w[2], w[3]), pair_hi(w[4], w[5]),     \
                              pair_hi(w[6], w[7]));                                              \
    _Pragma("unroll") for (int n = 0; n < NQ; ++n) _Pragma("unroll") for (int p = 0; p < PARTS; ++p) { \
      acc[n][e][2 * B] = mfma(v0, pr[n][p], acc[n][e][2 * B]);                                   \
      acc[n][e][2 * B + 1] = mfma(v1, pr[n][p], acc[n][e][2 * B + 1]);                           \
    }                                                                                            \
  }
            ARD_PAIR(0) ARD_PAIR(1) ARD_PAIR(2) ARD_PAIR(3)
#undef ARD_PAIR
          }
        }
        if (kLate) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < kSets; ++e) now.v[u][e] = next.v[u][e], now.vs[u][e] = next.vs[u][e];
        } else {
          now = next;
        }
        both = both_next;
      }

      // Join the waves: every wave's sums in units of the workgroup's maximum, added through LDS.
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        l[n] = row_sum(l[n]);
        nan_groups[n] = row_or(nan_groups[n]);
        if (g == 0) stat_m[wave][n * 16 + c] = m[n], stat_l[wave][n * 16 + c] = l[n];
      }
      __syncthreads();
      const int seg_per = NC;  // eight elements a thread
      const bool alone = parts == 1;
      auto finish = [&](int r, int seg, f32x4 o0, f32x4 o1, float top, float rl) {
        const int i = i0 + token_of(r), head = run.head * group + row0 + r - i * group;
        finish_row<DT>(a, me.q0 + i, head, seg, o0, o1, top, rl);
      };
      const ar::rsrc_t part = ar::make_rsrc(args.part, args.part_bytes);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float top = stat_m[0][n * 16 + c];
#pragma unroll
        for (int w = 1; w < kAttnWaves; ++w) top = fmaxf(top, stat_m[w][n * 16 + c]);
        const float f = exp2_fast(m[n] - top);
        if (__any(nan_groups[n] != 0)) {
#pragma unroll
          for (int e = 0; e < kSets; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (nan_groups[n] >> ((e * 16 + g * 4 + i) >> 2) & 1) {
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[n][e][j][i] = __uint_as_float(0x7FC00000u);
              }
        }
        float* mine = join + (wave * 16 + c) * kPitch;
#pragma unroll
        for (int e = 0; e < kSets; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int chunk = e * 16 + g * 4 + i;
            if (chunk < NC) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                f32x4 v;
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = acc[n][e][4 * h + j][i] * f;
                *reinterpret_cast<f32x4*>(mine + chunk * 8 + 4 * h) = v;
              }
            }
          }
        __syncthreads();
        for (int x = tid; x < 16 * seg_per; x += kAttnThreads) {
          const int r = x / seg_per, seg = x - r * seg_per, row = row0 + n * 16 + r;
          f32x4 o0 = {0, 0, 0, 0}, o1 = {0, 0, 0, 0};
          float rm = stat_m[0][n * 16 + r], rl = 0.0f;
#pragma unroll
          for (int w = 1; w < kAttnWaves; ++w) rm = fmaxf(rm, stat_m[w][n * 16 + r]);
#pragma unroll
          for (int w = 0; w < kAttnWaves; ++w) {
            const float* p = join + (w * 16 + r) * kPitch + seg * 8;
            o0 += *reinterpret_cast<const f32x4*>(p);
            o1 += *reinterpret_cast<const f32x4*>(p + 4);
            rl += stat_l[w][n * 16 + r] * exp2_fast(stat_m[w][n * 16 + r] - rm);
          }
          if (row >= rows) continue;
          if (!alone) {
            const uint32_t at = static_cast<uint32_t>((2 * w + (before == 0)) * R + n * 16 + r);
            ar::st16<ar::kCoh>(part, (at * D + seg * 8) * 4, __builtin_bit_cast(u32x4, o0));
            ar::st16<ar::kCoh>(part, (at * D + seg * 8 + 4) * 4, __builtin_bit_cast(u32x4, o1));
            if (seg == 0)
              ar::st8<ar::kCoh>(part, args.stats_at + at * 8, u32x2{__float_as_uint(rm), __float_as_uint(rl)});
            continue;
          }
          finish(n * 16 + r, seg, o0, o1, rm, rl);
        }
        if (n + 1 < NQ) __syncthreads();
      }
      if (!alone && arrive(args.arrived + first_wg, parts, &last))
        join_parts<D, R, 8>(part, args.stats_at, first_wg, parts, min(R, rows - row0), join, finish);
    }
    if (run.left <= 0) return;
    next_job<R>(args, run, me);
    if (run.left <= 0) return;
    __syncthreads();  // the next job's joins use the same LDS
  }
}

}  // namespace ard
