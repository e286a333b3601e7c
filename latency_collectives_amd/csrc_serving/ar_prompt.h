// Attention over packed prompts (gfx950): causal, grouped heads, each request's keys and values as the
// projection left them.
//
// Mathematics, split of the work and joins as in csrc_decode/ar_decode_attn_rows.h: products transposed, a running maximum, a
// workgroup's four waves on 16 * NQ rows each and on the same tokens. Keys and values come through LDS, a
// round (SUB units of 32 tokens) ahead, in the order of the products' operands:
//
//   bfloat16   S^T = K Q^T in 16x16x32 products; an operand of K is 16 bytes of a row as they are. O^T += V^T P^T:
//              a lane loads four elements of eight tokens and pairs tokens with one permute a word.
//   binary32   in 16x16x4 products, whose operands are single values: K in fours along a row, V as it lies.
//
// Keys and values past a request's end read as zero by the buffer's bounds and are masked like any other.
#pragma once

#include "../csrc_decode/ar_decode_attn_rows.h"
#include "ar_kv8.h"

namespace ard {

struct PromptArgs {
  ar_prompt_attention_args a;
  struct {
    int heads;
  } cache;
  int group;
  float per_group;
  uint32_t most_seen, unit, runs;
  int unit_shift, tile_shift, job_units;
  float scale_log2;  // its absolute value for bfloat16
  uint32_t q_sign;   // there: its sign, on two bfloat16
  int tile_tokens;
  uint8_t* part;
  uint32_t part_bytes, stats_at;
  uint32_t* arrived;
};

struct PromptKernel {
  void (*fn)(PromptArgs);
  int fill, rows;
};
PromptKernel select_prompt_bf16(int head_dim);
PromptKernel select_prompt_f32(int head_dim);

template <int R>
__device__ __forceinline__ Series series_of(const PromptArgs& args, int b) {
  Series c = {0, 0, 0, 0, 1, 0.0};
  if (b < args.a.nreq) {
    const int at = args.a.q_start[b], to = args.a.q_start[b + 1];
    c.q0 = min(max(at, 0), args.a.ntokens);
    c.m = c.kv = max(min(to, args.a.ntokens), c.q0) - c.q0;  // an end may be any number
    c.tiles = static_cast<int>((static_cast<uint32_t>(c.m) * static_cast<uint32_t>(args.group) + R - 1) / R);
    auto units = [&](int seen) {
      return ((min(static_cast<uint32_t>(seen), args.most_seen) + args.unit - 1) >> args.unit_shift) + args.job_units;
    };
    c.first = units(min(args.tile_tokens, c.m));
    if (c.tiles > 1) c.half_slope = static_cast<double>(units(c.m) - c.first) / (2 * (c.tiles - 1));
  }
  return c;
}

// A request's keys or values of one head from token t0 on, as a buffer that ends with its last token; what lies
// beyond reads as zero. A round's offsets stay below 2^30 (the host limits the stride).
__device__ __forceinline__ ar::rsrc_t rows_from(const uint8_t* base, int64_t row_bytes, int t0, int tokens, int width) {
  const int left = tokens - t0;
  const int64_t bytes = left > 0 ? (left - 1) * row_bytes + width : 0;
  return ar::make_rsrc(ar::uniform_ptr(base + (left > 0 ? t0 * row_bytes : 0)),
                       static_cast<uint32_t>(uniform(static_cast<int>(min(bytes, int64_t(0x7FFFFFFF))))));
}

// A round of tokens on its way into LDS: what each of four waves loads of it, and where it goes.
template <int DT, int D, int SUB>
struct Stage;

template <int D, int SUB>
struct Stage<DT_BF16, D, SUB> {
  static constexpr int kSteps = D / 32, kSets = (D + 63) / 64;
  static constexpr int kHalves = SUB * 2 / kAttnWaves;                       // 16 tokens of keys, of a wave
  static constexpr int kItems = (SUB * kSets + kAttnWaves - 1) / kAttnWaves;  // (unit, set) of values, of a wave
  static_assert(SUB * 2 % kAttnWaves == 0);
  struct Lds {
    u32x4 keys[SUB * 2][kSteps][64];
    u32x4 values[SUB][kSets][4][64];
  };
  u32x4 k[kHalves][kSteps];
  u32x2 v[kItems][8];

  __device__ void load(ar::rsrc_t kr, ar::rsrc_t vr, uint32_t k_row, uint32_t v_row, int wave, int c, int g) {
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        k[h][s] = ar::ld16<ar::kPlain>(kr, ((wave * kHalves + h) * 16 + c) * k_row + s * 64 + g * 16);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int item = min(wave * kItems + i, SUB * kSets - 1), unit = item / kSets, set = item - unit * kSets;
#pragma unroll
      for (int t = 0; t < 8; ++t)  // lanes beyond the row repeat its last elements
        v[i][t] = ar::ld8<ar::kPlain>(vr, (unit * 32 + (t >> 2) * 16 + g * 4 + (t & 3)) * v_row + min(set * 64 + c * 4, D - 4) * 2);
    }
  }
  __device__ bool odd() const {  // a value that is not finite
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
      for (int t = 0; t < 8; ++t) bad |= finite_only(v[i][t].x) != v[i][t].x || finite_only(v[i][t].y) != v[i][t].y;
    return bad;
  }
  __device__ void store(Lds& to, int wave, int lane) const {
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int s = 0; s < kSteps; ++s) to.keys[wave * kHalves + h][s][lane] = k[h][s];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int item = wave * kItems + i;
      if (item >= SUB * kSets) break;
      const int unit = item / kSets, set = item - unit * kSets;
      const u32x2* x = v[i];
      to.values[unit][set][0][lane] = u32x4{pair_lo(x[0].x, x[1].x), pair_lo(x[2].x, x[3].x), pair_lo(x[4].x, x[5].x), pair_lo(x[6].x, x[7].x)};
      to.values[unit][set][1][lane] = u32x4{pair_hi(x[0].x, x[1].x), pair_hi(x[2].x, x[3].x), pair_hi(x[4].x, x[5].x), pair_hi(x[6].x, x[7].x)};
      to.values[unit][set][2][lane] = u32x4{pair_lo(x[0].y, x[1].y), pair_lo(x[2].y, x[3].y), pair_lo(x[4].y, x[5].y), pair_lo(x[6].y, x[7].y)};
      to.values[unit][set][3][lane] = u32x4{pair_hi(x[0].y, x[1].y), pair_hi(x[2].y, x[3].y), pair_hi(x[4].y, x[5].y), pair_hi(x[6].y, x[7].y)};
    }
  }
};

template <int D, int SUB>
struct Stage<DT_F32, D, SUB> {
  static constexpr int kSteps = D / 16, kSets = (D + 63) / 64;  // a step: four products along a row
  static constexpr int kKeys = SUB * 2 * kSteps / kAttnWaves;   // (half, step) of a wave
  static constexpr int kRows = SUB * 32 / kAttnWaves;           // tokens of values, of a wave
  static constexpr int kItems = kRows * D / 256;                // 64 lanes, four elements each
  static_assert(SUB * 2 * kSteps % kAttnWaves == 0 && kRows * D % 256 == 0);
  struct Lds {
    f32x4 keys[SUB * 2][kSteps][64];
    f32x4 values[SUB * 32][D / 4];
  };
  f32x4 k[kKeys];
  f32x4 v[kItems];

  __device__ void load(ar::rsrc_t kr, ar::rsrc_t vr, uint32_t k_row, uint32_t v_row, int wave, int c, int g) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int x = wave * kKeys + i, half = x / kSteps, s = x - half * kSteps;
      k[i] = __builtin_bit_cast(f32x4, ar::ld16<ar::kPlain>(kr, (half * 16 + c) * k_row + s * 64 + g * 16));
    }
    const int lane = g * 16 + c;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int x = i * 64 + lane, row = x / (D / 4);
      v[i] = __builtin_bit_cast(f32x4, ar::ld16<ar::kPlain>(vr, (wave * kRows + row) * v_row + (x - row * (D / 4)) * 16));
    }
  }
  __device__ bool odd() const {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) bad |= !(fabsf(v[i][j]) < INFINITY);
    return bad;
  }
  __device__ void store(Lds& to, int wave, int lane) const {
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int x = wave * kKeys + i, half = x / kSteps, s = x - half * kSteps;
      to.keys[half][s][lane] = k[i];
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int x = i * 64 + lane, row = x / (D / 4);
      to.values[wave * kRows + row][x - row * (D / 4)] = v[i];
    }
  }
};

__device__ __forceinline__ f32x4 mfma1(float a, float b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

template <int DT, int D, int NQ, int SUB, int OCC>
__global__ __launch_bounds__(kAttnThreads, OCC) void prompt_attention(PromptArgs args) {
  constexpr int RW = 16 * NQ, R = RW * kAttnWaves;
  constexpr bool kBf16 = DT == DT_BF16;
  constexpr int ES = kBf16 ? 2 : 4;
  typedef Stage<DT, D, SUB> Round;
  constexpr int kSteps = Round::kSteps, kSets = Round::kSets;
  typedef typename std::conditional<kBf16, bf16x8, f32x4>::type Q;  // a lane's elements of a step
  __shared__ typename Round::Lds tokens[2];
  __shared__ u32x4 any_odd[2];  // a word a wave
  __shared__ int last;

  const ar_prompt_attention_args& a = args.a;
  // consecutive runs on one XCD: workgroups go to the eight in turn
  const int w = (blockIdx.x & 7) * (args.runs >> 3) + (blockIdx.x >> 3);
  Run run;
  Series me;
  int span;
  if (!find_rows<R>(args, w, run, me, span)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int group = args.group;
  const int64_t k_row = a.k_token * ES, v_row = a.v_token * ES;
  const ar::rsrc_t part = ar::make_rsrc(args.part, args.part_bytes);

  for (;;) {
    const int rows = me.m * group;
    const int row0 = run.tile * R;
    const int i0 = uniform(static_cast<uint32_t>(row0) / static_cast<uint32_t>(group)), rem0 = row0 - i0 * group;
    // token of row row0 + r: rem0 + r is below 2^17, exact in binary32
    auto token_of = [&](int r) { return static_cast<int>((rem0 + r + 0.5f) * args.per_group); };
    const int i1 = i0 + uniform(token_of(min(R, rows - row0) - 1));
    const int end = i1 + 1;
    const int begin = a.window > 0 ? max(window_start(i0, a.window), 0) & ~31 : 0;
    const int ntiles = (end - begin + 31) >> 5;
    const int nunits = (ntiles + (1 << args.tile_shift) - 1) >> args.tile_shift;
    const int taken = min(run.left, span - run.at);
    const bool ends = run.at + taken == span;  // the last part takes what the series left out
    const int t_first = run.at << args.tile_shift;
    const int t_last = ends ? ntiles : min((run.at + taken) << args.tile_shift, ntiles);
    run.left -= taken;
    int before = 0, first_units = taken;
    if (run.at > 0) {
      before = uniform(static_cast<uint32_t>(run.at + run.per - 1) / static_cast<uint32_t>(run.per));
      first_units = run.at - (before - 1) * run.per;
    }
    const int first_wg = w - before;
    int parts = 1;
    if (min(nunits, span) > first_units)
      parts = 1 + uniform(static_cast<uint32_t>(min(nunits, span) - first_units + run.per - 1) /
                          static_cast<uint32_t>(run.per));
    if (run.at == 0 || t_first < ntiles) {
      const uint8_t* keys = static_cast<const uint8_t*>(a.k) + me.q0 * k_row + run.head * a.k_head * ES;
      const uint8_t* vals = static_cast<const uint8_t*>(a.v) + me.q0 * v_row + run.head * a.v_head * ES;
      const int t_begin = begin + t_first * 32, t_end = min(begin + t_last * 32, end);
      Round next;
      auto load = [&](int t) {
        next.load(rows_from(keys, k_row, t, end, D * ES), rows_from(vals, v_row, t, end, D * ES),
                  static_cast<uint32_t>(k_row), static_cast<uint32_t>(v_row), wave, c, g);
      };
      // Rounds that some row sees in part: from the first row's end on, and up to the last one's window.
      const int odd_begin = a.window > 0 ? window_start(i1, a.window) : 0;
      auto store = [&](int buf, int t) {
        next.store(tokens[buf], wave, lane);
        bool some = false;
        if (t + SUB * 32 > i0 + 1 || t < odd_begin) some = __any(next.odd());
        if (lane == 0) reinterpret_cast<uint32_t*>(&any_odd[buf])[wave] = some;
      };
      if (t_begin < t_end) load(t_begin);

      // This wave's rows.
      const int mine0 = row0 + wave * RW;
      int hi[NQ], lo[NQ];
      Q q[NQ][kSteps];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        // rows past the last repeat it
        const int r = min(wave * RW + n * 16 + c, rows - 1 - row0), i = i0 + token_of(r);
        hi[n] = i + 1;
        lo[n] = a.window > 0 ? window_start(i, a.window) : 0;
        const int64_t at = static_cast<int64_t>(me.q0 + i) * a.q_token +
                           static_cast<int64_t>(run.head * group + row0 + r - i * group) * a.q_head;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          if constexpr (kBf16)
            q[n][s] = __builtin_bit_cast(
                bf16x8, *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.q) + at + s * 32 + g * 8) ^ args.q_sign);
          else
            q[n][s] = *reinterpret_cast<const f32x4*>(static_cast<const float*>(a.q) + at + s * 16 + g * 4);
        }
      }
      const int i_first = i0 + token_of(min(wave * RW, rows - 1 - row0));
      const int i_last = i0 + token_of(min(wave * RW + RW, rows - row0) - 1);
      const int my_end = uniform(mine0 < rows ? min(i_last + 1, t_end) : 0);
      // Units from here on need masks: the first row's end, the last row's window.
      const int whole_end = uniform(i_first + 1);
      const int whole_begin = uniform(a.window > 0 ? window_start(i_last, a.window) : 0);
      const int my_begin = uniform(a.window > 0 ? max(window_start(i_first, a.window), 0) : 0);

      f32x4 acc[NQ][kSets][4];  // [i]: element 64 e + 16 g + 4 i + j of row c
      float m[NQ], l[NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        m[n] = kLowest, l[n] = 0.0f;
#pragma unroll
        for (int e = 0; e < kSets; ++e)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[n][e][j] = f32x4{0, 0, 0, 0};
      }

      int buf = 0;
      if (t_begin < t_end) store(0, t_begin);
      __syncthreads();
      for (int tr = t_begin; tr < t_end; tr += SUB * 32) {
        const bool more = tr + SUB * 32 < t_end;
        const u32x4 some_odd = any_odd[buf];
        const bool round_odd = uniform(some_odd[0] | some_odd[1] | some_odd[2] | some_odd[3]) != 0;
        if (more) load(tr + SUB * 32);
#pragma unroll 1
        for (int sub = 0; sub < SUB; ++sub) {
          const int t0 = tr + sub * 32;
          if (t0 >= my_end || t0 + 32 <= my_begin) continue;
          const bool masked = t0 + 32 > whole_end || t0 < whole_begin;
          auto sees = [&](int n, int u, int i) {
            const int t = t0 + u * 16 + g * 4 + i;
            return t < hi[n] && t >= lo[n];
          };
          auto values_of = [&](int j) {  // bfloat16: the operand of elements 64 (j / 4) + 4 c + j % 4
            if constexpr (kBf16) return tokens[buf].values[sub][j >> 2][j & 3][lane];
            else return u32x4{};
          };
          auto value4 = [&](int u, int i, int e) {  // binary32: four elements of token 4 g + i of half u
            if constexpr (kBf16) return f32x4{};
            else return tokens[buf].values[sub * 32 + u * 16 + g * 4 + i][min(e * 16 + c, D / 4 - 1)];
          };
          const bool scrub = masked && round_odd;  // infinities and NaN of tokens that only some rows see
          if (scrub) {
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              const bf16x8 visible = visible_of([&](int u, int i) { return sees(n, u, i); });
              if constexpr (kBf16) {
#pragma unroll
                for (int j = 0; j < 4 * kSets; ++j) {
                  add_infinite(values_of(j), visible, acc[n][j >> 2][j & 3]);
                  __builtin_amdgcn_sched_barrier(0);
                }
              } else {
#pragma unroll
                for (int e = 0; e < kSets; ++e) {
                  f32x4 up[4], down[4];
#pragma unroll
                  for (int j = 0; j < 4; ++j) up[j] = down[j] = f32x4{0, 0, 0, 0};
#pragma unroll
                  for (int x = 0; x < 8; ++x) {
                    const f32x4 y = value4(x >> 2, x & 3, e);
                    const float one = sees(n, x >> 2, x & 3) ? 1.0f : 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                      up[j] = mfma1(y[j] <= 3.4028235e38f ? 0.0f : 1.0f, one, up[j]);
                      down[j] = mfma1(y[j] >= -3.4028235e38f ? 0.0f : 1.0f, one, down[j]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                  }
#pragma unroll
                  for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                      if (up[j][i] > 0.0f) acc[n][e][j][i] += INFINITY;
                      if (down[j][i] > 0.0f) acc[n][e][j][i] -= INFINITY;
                    }
                }
              }
            }
          }
          // Scores.
          __builtin_amdgcn_s_setprio(1);
          f32x4 s[NQ][2];
#pragma unroll
          for (int n = 0; n < NQ; ++n) s[n][0] = s[n][1] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
              const auto kk = __builtin_bit_cast(Q, tokens[buf].keys[sub * 2 + u][i][lane]);
#pragma unroll
              for (int n = 0; n < NQ; ++n) {
                if constexpr (kBf16) {
                  s[n][u] = mfma(kk, q[n][i], s[n][u]);
                } else {
#pragma unroll
                  for (int j = 0; j < 4; ++j) s[n][u] = mfma1(kk[j], q[n][i][j], s[n][u]);
                }
              }
            }
          __builtin_amdgcn_s_setprio(0);
          if (!kBf16)
#pragma unroll
            for (int n = 0; n < NQ; ++n) s[n][0] *= args.scale_log2, s[n][1] *= args.scale_log2;
          if (masked) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (!sees(n, u, i)) s[n][u][i] = -INFINITY;
          }
          // The first operands of the second product, under way with the probabilities.
          constexpr int AHEAD = 4;
          u32x4 vv[AHEAD];
          if constexpr (kBf16) {
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) vv[j] = values_of(j);
            __builtin_amdgcn_sched_barrier(0);
          }
          // Probabilities.
          bf16x8 pr[NQ];
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            float top = s[n][0][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top = fmaxf(top, s[n][i >> 2][i & 3]);
            if (kBf16) top *= args.scale_log2;
            if (__any(top > m[n] + 8.0f)) {
              const float to = fmaxf(m[n], row_max(top));
              const float f = exp2_fast(m[n] - to);
              m[n] = to;
              l[n] *= f;
#pragma unroll
              for (int e = 0; e < kSets; ++e)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[n][e][j] *= f;
            }
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              x[i] = exp2_fast(kBf16 ? fmaf(s[n][i >> 2][i & 3], args.scale_log2, -m[n]) : s[n][i >> 2][i & 3] - m[n]);
              l[n] += x[i];
            }
            if constexpr (kBf16) split<1>(x, &pr[n]);
            else
#pragma unroll
              for (int i = 0; i < 8; ++i) s[n][i >> 2][i & 3] = x[i];
          }
          // Values.
          if constexpr (kBf16) {
#pragma unroll
            for (int j = 0; j < 4 * kSets; ++j) {
              u32x4 x = vv[j % AHEAD];
              if (j + AHEAD < 4 * kSets) vv[j % AHEAD] = values_of(j + AHEAD);
              if (scrub)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = finite_only(x[i]);
#pragma unroll
              for (int n = 0; n < NQ; ++n) acc[n][j >> 2][j & 3] = mfma(__builtin_bit_cast(bf16x8, x), pr[n], acc[n][j >> 2][j & 3]);
            }
          } else {
#pragma unroll
            for (int x = 0; x < 8; ++x)
#pragma unroll
              for (int e = 0; e < kSets; ++e) {
                f32x4 y = value4(x >> 2, x & 3, e);
                if (scrub)
#pragma unroll
                  for (int j = 0; j < 4; ++j) y[j] = fabsf(y[j]) < INFINITY ? y[j] : 0.0f;
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                  for (int j = 0; j < 4; ++j) acc[n][e][j] = mfma1(y[j], s[n][x >> 2][x & 3], acc[n][e][j]);
              }
          }
        }
        if (more) store(buf ^ 1, tr + SUB * 32);
        buf ^= 1;
        __syncthreads();
      }

      // This wave's rows are its own: out, or into the workspace.
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        l[n] = row_sum(l[n]);
        const int r = wave * RW + n * 16 + c;
        if (row0 + r < rows) {
          const int i = i0 + token_of(r), head = run.head * group + row0 + r - i * group;
          const int64_t token = me.q0 + i;
          const float f = parts > 1 ? 1.0f : l[n] == 0.0f ? 0.0f : 1.0f / l[n];
          const uint32_t at = static_cast<uint32_t>((2 * w + (before == 0)) * R + r);
#pragma unroll
          for (int e = 0; e < kSets; ++e) {
            if (e * 64 + g * 16 >= D) continue;  // a lane's sixteen elements: all in the row or none
            float o[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] = acc[n][e][x & 3][x >> 2] * f;
            const int from = e * 64 + g * 16;
            const int64_t to = token * a.o_token + head * a.o_head + from;
            if (parts > 1) {
#pragma unroll
              for (int x = 0; x < 16; x += 4)
                ar::st16<ar::kCoh>(part, (at * D + from + x) * 4,
                                   u32x4{__float_as_uint(o[x]), __float_as_uint(o[x + 1]), __float_as_uint(o[x + 2]),
                                         __float_as_uint(o[x + 3])});
            } else if constexpr (kBf16) {
              u32x4* p = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + to);
#pragma unroll
              for (int x = 0; x < 16; x += 8)
                p[x / 8] = u32x4{ar::bf16x2_rne(o[x], o[x + 1]), ar::bf16x2_rne(o[x + 2], o[x + 3]),
                                 ar::bf16x2_rne(o[x + 4], o[x + 5]), ar::bf16x2_rne(o[x + 6], o[x + 7])};
            } else {
              f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + to);
#pragma unroll
              for (int x = 0; x < 16; x += 4) p[x / 4] = f32x4{o[x], o[x + 1], o[x + 2], o[x + 3]};
            }
          }
          if (g == 0) {
            if (parts > 1)
              ar::st8<ar::kCoh>(part, args.stats_at + at * 8, u32x2{__float_as_uint(m[n]), __float_as_uint(l[n])});
            else if (a.lse != nullptr)
              a.lse[token * a.q_heads + head] = l[n] == 0.0f ? -INFINITY : (m[n] + log2f(l[n])) * 0.6931471805599453f;
          }
        }
      }
      if (parts > 1) {
        auto finish = [&](int r, int seg, f32x4 o0, f32x4 o1, float top, float rl) {
          const int i = i0 + token_of(r), head = run.head * group + row0 + r - i * group;
          finish_row<DT>(a, me.q0 + i, head, seg, o0, o1, top, rl);
        };
        if (arrive(args.arrived + first_wg, parts, &last)) {
          const int real = min(R, rows - row0);
          if (parts == 2) join_few<D, R, 2, 4>(part, args.stats_at, first_wg, parts, real, finish);
          else if (parts <= 4) join_few<D, R, 4, 2>(part, args.stats_at, first_wg, parts, real, finish);
          else join_parts<D, R, 8>(part, args.stats_at, first_wg, parts, real, reinterpret_cast<float*>(tokens), finish);
        }
      }
    }
    if (run.left <= 0) return;
    // The next job of the run.
    run.at = 0;
    if (++run.tile == me.tiles) {
      run.tile = 0;
      if (++run.head == args.cache.heads) {
        run.head = 0;
        do {
          if (++run.request >= a.nreq) return;  // only if starts change under the call
          me = series_of<R>(args, run.request);
          me.tiles = uniform(me.tiles);
        } while (me.tiles == 0);
      }
    }
    span = uniform(me.below(run.tile + 1) - me.below(run.tile));
    __syncthreads();  // the next job uses the same LDS
  }
}

}  // namespace ard
