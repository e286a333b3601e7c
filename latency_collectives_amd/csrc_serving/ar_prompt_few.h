// Attention over packed prompts where rows are few (gfx950): a tile of 16 rows a workgroup, its four waves on different
// tokens.
//
// Such a call is bound by latency: what stands one after the other is the launch, the starts, the first keys and values, a
// wave's units, the join. So there is no split between workgroups and no workspace; a workgroup finds its tile by one scan
// over the starts; a wave takes every fourth unit, straight from memory into the operands' registers, and the four sums
// meet in LDS. A unit's registers take the next one's keys and values as soon as they have been used: with a second set of
// them a compute unit held fewer workgroups (head of 192: 20.0 us for seven prompts of up to 301 tokens, 14.0 so; 500 of up to 5,
// head of 128, 9.4 and 6.6).
//
//   bfloat16   a unit is 32 tokens; values: four elements of eight tokens a lane, tokens paired by one permute a word
//   binary32   a unit is 16 tokens; values: four elements of a token a lane, as the 16x16x4 products take them
//
// One prompt of 301 tokens, 8 query heads on one kv head of 128, bfloat16: 7.8 us, 16.3 by the kernels for many rows.
#pragma once

#include "ar_prompt.h"

namespace ard {

template <int DT, int D>
struct FewUnit {  // a lane's share of a unit, as loaded
  static constexpr bool kBf16 = DT == DT_BF16;
  static constexpr int kSteps = kBf16 ? D / 32 : D / 16, kSets = (D + 63) / 64;
  static constexpr int U = kBf16 ? 2 : 1;  // times 16 tokens
  typedef typename std::conditional<kBf16, u32x2, u32x4>::type V;
  u32x4 k[U][kSteps];
  V v[4 * U][kSets];  // [u * 4 + i]: token 16 u + 4 g + i
};

// At voffset + soffset of the buffer, the second the same for all lanes; both count for its end.
template <class T>
__device__ __forceinline__ T row_at(ar::rsrc_t from, uint32_t voffset, uint32_t soffset) {
  if constexpr (sizeof(T) == 16) return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b128(from, voffset, soffset, 0));
  else return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b64(from, voffset, soffset, 0));
}

// Tile `x` from the last; tells whether there is one a grid further, which takes requests that overlap: the grid (`runs`)
// has the tiles of tokens that each belong to one request.
template <int DT, int D>
__device__ __forceinline__ bool few_tile(const PromptArgs& args, uint32_t x) {
  constexpr int R = 16;
  constexpr bool kBf16 = DT == DT_BF16;
  constexpr int ES = kBf16 ? 2 : 4, NC = D / 8;
  typedef FewUnit<DT, D> Unit;
  typedef typename std::conditional<kBf16, bf16x8, f32x4>::type Q;
  constexpr int kSteps = Unit::kSteps, kSets = Unit::kSets, U = Unit::U, T = 16 * U;
  static_assert(offsets_fit(T));
  constexpr int kPitch = D + 4;  // LDS row: 16 rows' 16-byte accesses fall into different banks
  __shared__ float join[kAttnWaves * 16 * kPitch];
  __shared__ float stat_m[kAttnWaves][R], stat_l[kAttnWaves][R];
  __shared__ uint32_t tiles_in_all;

  const ar_prompt_attention_args& a = args.a;
  const int lane = thread_here() & 63, wave = uniform(thread_here() >> 6), c = lane & 15, g = lane >> 4;
  // The tile: a lane's requests lie side by side; where those are several, the lane's that has it then one a lane.
  uint32_t tile;
  PromptJob j;
  {
    const int each = (a.nreq + 63) >> 6;
    int q0, m;
    auto tiles_of = [&](int b) {
      const int x = min(b, a.nreq - 1);
      const int at = a.q_start[x], to = a.q_start[x + 1];
      q0 = min(max(at, 0), a.ntokens);
      m = b < a.nreq ? max(min(to, a.ntokens), q0) - q0 : 0;
      return (static_cast<uint32_t>(m) * static_cast<uint32_t>(args.group) + R - 1) / R;
    };
    uint32_t tiles = 0;
#pragma unroll 4
    for (int i = 0; i < each; ++i) tiles = __builtin_elementwise_add_sat(tiles, tiles_of(lane * each + i));
    uint32_t upto = wave_scan(tiles);
    const uint32_t all = static_cast<uint32_t>(lane_value(upto, 63));
    if (x >= all || all >> 8 > args.runs) return false;  // an end to what overlaps can ask for
    if (threadIdx.x == 0) tiles_in_all = all;  // kept there: the loop needs the registers
    tile = all - 1 - x;  // a prompt's last tiles see most: they go first
    int who = __builtin_ctzll(__ballot(upto > tile));
    tile -= static_cast<uint32_t>(lane_value(upto - tiles, who));
    if (each > 1) {
      for (int b = who * each;; b += 64) {
        tiles = tiles_of(b + lane);
        upto = wave_scan(tiles);
        if (__ballot(upto > tile) != 0) break;
        tile -= static_cast<uint32_t>(lane_value(upto, 63));
        if (b + 64 >= a.nreq) return false;  // only if starts change under the call
      }
      who = __builtin_ctzll(__ballot(upto > tile));
      tile -= static_cast<uint32_t>(lane_value(upto - tiles, who));
    }
    j.q0 = lane_value(q0, who);
    j.rows = lane_value(m, who) * args.group;
  }
  j.head = blockIdx.y, j.group = args.group, j.per_group = args.per_group, j.window = a.window;
  j.row0 = uniform(static_cast<int>(tile * R));
  j.i0 = uniform(static_cast<uint32_t>(j.row0) / static_cast<uint32_t>(j.group)), j.rem0 = j.row0 - j.i0 * j.group;
  const int last = min(R, j.rows - j.row0) - 1;
  j.i1 = j.i0 + uniform(j.token_of(last));
  const int end = j.i1 + 1, begin = a.window > 0 ? max(window_start(j.i0, a.window), 0) & ~31 : 0;
  j.k_row = a.k_token * ES, j.v_row = a.v_token * ES;
  const uint8_t* keys = static_cast<const uint8_t*>(a.k) + j.q0 * j.k_row + j.head * a.k_head * ES;
  const uint8_t* vals = static_cast<const uint8_t*>(a.v) + j.q0 * j.v_row + j.head * a.v_head * ES;

  // Places of a lane, and what is the same for all of them beside.
  const uint32_t k_row = static_cast<uint32_t>(j.k_row), v_row = static_cast<uint32_t>(j.v_row);
  const uint32_t k_off = c * k_row + g * 16;
  uint32_t v_off[kSets];
#pragma unroll
  for (int e = 0; e < kSets; ++e) v_off[e] = g * 4 * v_row + min(e * 64 + c * 4, D - 4) * ES;  // lanes beyond the row repeat its last elements
  auto load_keys = [&](int t0, Unit& x) {
    const ar::rsrc_t kr = rows_from(keys, j.k_row, t0, end, D * ES);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int s = 0; s < kSteps; ++s) x.k[u][s] = row_at<u32x4>(kr, k_off, u * 16 * k_row + s * 64);
  };
  auto load_values = [&](int t0, Unit& x) {
    const ar::rsrc_t vr = rows_from(vals, j.v_row, t0, end, D * ES);
#pragma unroll
    for (int t = 0; t < 4 * U; ++t)
#pragma unroll
      for (int e = 0; e < kSets; ++e) x.v[t][e] = row_at<typename Unit::V>(vr, v_off[e], ((t >> 2) * 16 + (t & 3)) * v_row);
  };
  Unit now;
  int t0 = begin + wave * T;
  if (t0 < end) load_keys(t0, now), load_values(t0, now);

  // The rows, the same for every wave.
  const int r = min(c, last), i = j.i0 + j.token_of(r);
  const int hi = i + 1, lo = a.window > 0 ? window_start(i, a.window) : 0;
  const int whole_end = j.i0 + 1, whole_begin = a.window > 0 ? window_start(j.i1, a.window) : 0;
  Q q[kSteps];
  {
    const int64_t at = static_cast<int64_t>(j.q0 + i) * a.q_token +
                       static_cast<int64_t>(j.head * j.group + j.row0 + r - i * j.group) * a.q_head;
    const uint8_t* x = static_cast<const uint8_t*>(a.q) + at * ES + g * 16;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const u32x4 y = *reinterpret_cast<const u32x4*>(x + s * 64);
      if constexpr (kBf16) q[s] = __builtin_bit_cast(Q, y ^ args.q_sign);
      else q[s] = __builtin_bit_cast(Q, y);
    }
  }

  f32x4 acc[kSets][4];  // [k]: element 64 e + 16 g + 4 k + j of row c
  float m = kLowest, l = 0.0f;
#pragma unroll
  for (int e = 0; e < kSets; ++e)
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[e][k] = zeros_here();

#pragma unroll 1
  for (; t0 < end; t0 += T * kAttnWaves) {
    // Scores.
    f32x4 s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const Q kk = __builtin_bit_cast(Q, now.k[u][k]);
        if constexpr (kBf16) {
          s[u] = mfma(kk, q[k], s[u]);
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x) s[u] = mfma1(kk[x], q[k][x], s[u]);
        }
      }
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] *= args.scale_log2;
    // The next unit's keys into their registers, as its values below.
    if (t0 + T * kAttnWaves < end) load_keys(t0 + T * kAttnWaves, now);
    auto sees = [&](int u, int x) {
      const int t = t0 + u * 16 + (thread_here() >> 4 & 3) * 4 + x;
      return t < hi && t >= lo;
    };
    // bfloat16: the operand of elements 64 e + 4 c + k.
    auto value_of = [&](int e, int k) {
      u32x4 w = {0, 0, 0, 0};
      if constexpr (kBf16) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const u32x2 v0 = now.v[2 * x][e], v1 = now.v[2 * x + 1][e];
          w[x] = k == 0 ? pair_lo(v0.x, v1.x) : k == 1 ? pair_hi(v0.x, v1.x) : k == 2 ? pair_lo(v0.y, v1.y) : pair_hi(v0.y, v1.y);
        }
      }
      return w;
    };
    if (t0 + T > whole_end || t0 < whole_begin) {
#pragma unroll
      for (int x = 0; x < 4 * U; ++x)
        if (!sees(x >> 2, x & 3)) s[x >> 2][x & 3] = -INFINITY;
      // Infinities and NaN that not all rows see: added for the rows that do, and taken out.
      bool odd = false;
#pragma unroll
      for (int t = 0; t < 4 * U; ++t)
#pragma unroll
        for (int e = 0; e < kSets; ++e)
#pragma unroll
          for (int x = 0; x < ES; ++x) {
            const uint32_t w = now.v[t][e][x];
            odd |= kBf16 ? finite_only(w) != w : (w & 0x7F800000u) == 0x7F800000u;
          }
      if (__any(odd)) {
#pragma unroll 1
        for (int t = t0; t < min(t0 + T, end); ++t) {
          if (t >= hi || t < lo) continue;
          const int from = (thread_here() >> 4 & 3) * 16;
#pragma unroll
          for (int e = 0; e < kSets; ++e) {
            if (64 * e + from >= D) continue;
            const u32x4* p = reinterpret_cast<const u32x4*>(vals + t * j.v_row + (64 * e + from) * ES);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              f32x4 y;
              if constexpr (kBf16) {
                const u32x2 w = reinterpret_cast<const u32x2*>(p)[x];
                y = f32x4{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
              } else {
                y = __builtin_bit_cast(f32x4, p[x]);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (!(fabsf(y[k]) < INFINITY)) acc[e][k][x] += y[k];
            }
          }
        }
#pragma unroll
        for (int t = 0; t < 4 * U; ++t)
#pragma unroll
          for (int e = 0; e < kSets; ++e)
#pragma unroll
            for (int x = 0; x < ES; ++x) {
              const uint32_t w = now.v[t][e][x];
              now.v[t][e][x] = kBf16 ? finite_only(w) : (w & 0x7F800000u) == 0x7F800000u ? 0 : w;
            }
      }
    }
    // Probabilities.
    float top = s[0][0];
#pragma unroll
    for (int x = 1; x < 4 * U; ++x) top = fmaxf(top, s[x >> 2][x & 3]);
    if (__any(top > m + 8.0f)) {
      const float to = fmaxf(m, row_max(top));
      const float f = shrink(m, to);
      m = to;
      l *= f;
#pragma unroll
      for (int e = 0; e < kSets; ++e)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[e][k] *= f;
    }
    float p[4 * U];
#pragma unroll
    for (int x = 0; x < 4 * U; ++x) {
      p[x] = exp2_fast(s[x >> 2][x & 3] - m);
      l += p[x];
    }
    // Values.
    if constexpr (kBf16) {
      bf16x8 pr;
      split<1>(p, &pr);
#pragma unroll
      for (int e = 0; e < kSets; ++e)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[e][k] = mfma(__builtin_bit_cast(bf16x8, value_of(e, k)), pr, acc[e][k]);
    } else {
#pragma unroll
      for (int t = 0; t < 4 * U; ++t)
#pragma unroll
        for (int e = 0; e < kSets; ++e)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[e][k] = mfma1(__uint_as_float(now.v[t][e][k]), p[t], acc[e][k]);
    }
    if (t0 + T * kAttnWaves < end) load_values(t0 + T * kAttnWaves, now);
  }

  {
    // Join the waves: every wave's sums in units of the workgroup's maximum, added through LDS.
    const int tid = thread_here(), c = tid & 15, g = tid >> 4 & 3;
    l = row_sum(l);
    if (g == 0) stat_m[wave][c] = m, stat_l[wave][c] = l;
    __syncthreads();
    float most = stat_m[0][c];
#pragma unroll
    for (int x = 1; x < kAttnWaves; ++x) most = fmaxf(most, stat_m[x][c]);
    const float f = exp2_fast(m - most);
    float* mine = join + (wave * 16 + c) * kPitch + g * 16;
#pragma unroll
    for (int e = 0; e < kSets; ++e)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (e * 64 + g * 16 + x * 4 >= D) continue;
        f32x4 v;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = acc[e][k][x] * f;
        *reinterpret_cast<f32x4*>(mine + e * 64 + x * 4) = v;
      }
    __syncthreads();
    for (int x = tid; x < 16 * NC; x += kAttnThreads) {
      const int row = x / NC, seg = x - row * NC;
      if (row > last) continue;
      f32x4 o0 = {0, 0, 0, 0}, o1 = {0, 0, 0, 0};
      float rm = stat_m[0][row], rl = 0.0f;
#pragma unroll
      for (int y = 1; y < kAttnWaves; ++y) rm = fmaxf(rm, stat_m[y][row]);
#pragma unroll
      for (int y = 0; y < kAttnWaves; ++y) {
        const float* from = join + (y * 16 + row) * kPitch + seg * 8;
        o0 += *reinterpret_cast<const f32x4*>(from);
        o1 += *reinterpret_cast<const f32x4*>(from + 4);
        rl += stat_l[y][row] * exp2_fast(stat_m[y][row] - rm);
      }
      const int token = j.i0 + j.token_of(row);
      finish_row<DT>(a, j.q0 + token, j.head * j.group + j.row0 + row - token * j.group, seg, o0, o1, rm, rl);
    }
  }
  return uniform(tiles_in_all) - x > args_here<PromptArgs>().runs;
}

template <int DT, int D>
__global__ __launch_bounds__(kAttnThreads, D > 192 ? 1 : D > 128 ? 2 : D > 64 ? 3 : 4) void prompt_attention_few(PromptArgs args) {
  // The first tile's code is its own: in the loop's it took 0.3 us longer (registers, a cold cache of instructions).
  if (__builtin_expect(!few_tile<DT, D>(args, blockIdx.x), 1)) return;
  for (uint32_t x = blockIdx.x + args.runs;; x += args.runs) {
    __syncthreads();  // the next tile uses the same LDS
    if (!few_tile<DT, D>(args_here<PromptArgs>(), x)) return;
  }
}

}  // namespace ard
