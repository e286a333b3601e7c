// Attention over the 8-bit paged cache for many query rows a request (prompt chunks), bfloat16.
//
// Mathematics, split of the work and joins as in csrc_decode/ar_decode_attn_rows.h; operands as in
// ar_kv8_attn.h. A workgroup's four waves hold 16 * NQ rows each and go through the same tokens
// together: each converts its operands of the keys in registers, in the shadow of the products; values
// become bfloat16 once a workgroup, each wave a quarter of a round's, through LDS.
#pragma once

#include "../csrc_decode/ar_decode_attn_rows.h"
#include "ar_kv8_attn.h"

namespace ard {

template <int D, int NQ, int OCC>
__global__ __launch_bounds__(kAttnThreads, OCC) void kv8_attention_rows(AttnArgs args) {
  constexpr int RW = 16 * NQ, R = RW * kAttnWaves;
  constexpr int kSteps = D / 32, kSets = (D + 63) / 64;
  constexpr int SPLIT = D > 128 ? 2 : 1;       // waves that share a unit's values
  constexpr int SUB = kAttnWaves / SPLIT;      // units of 32 tokens of a round
  constexpr int MINE = (kSets + SPLIT - 1) / SPLIT, OPS = 4 * MINE;  // sets, operands of a wave
  constexpr int TURNS = SPLIT == 1 ? 2 : 1;  // units in the loop's body: with two, keys stay where they are
  __shared__ u32x4 values[2][kAttnWaves][OPS][64];  // [buffer][unit, part of its sets][operand][lane]
  __shared__ u32x4 any_nan[2];  // a word a wave
  __shared__ int last;

  const ar_kv4_attention_args& a = args.a;
  // consecutive runs on one XCD: workgroups go to the eight in turn
  const int w = (blockIdx.x & 7) * (args.runs >> 3) + (blockIdx.x >> 3);
  Run run;
  Series me;
  int span;
  if (!find_rows<R>(args, w, run, me, span)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int group = args.group, shift = args.cache.page_shift;
  const int page = 1 << shift;
  const int num_pages = static_cast<int>(args.cache.num_pages);
  const uint32_t k_off = c * D + step_at<D>(0, g);
  const int my_set = wave % SPLIT * MINE, my_unit = wave / SPLIT;
  uint32_t v_off[MINE];
#pragma unroll
  for (int e = 0; e < MINE; ++e)  // lanes beyond the row repeat its last elements
    v_off[e] = page * D + g * (4 * D) + min((my_set + e) * 64 + c * 4, D - 4) * 4;
  const ar::rsrc_t part = ar::make_rsrc(args.part, args.part_bytes);

  for (;;) {
    const int rows = me.m * group;
    const int row0 = run.tile * R;
    const int i0 = uniform(static_cast<uint32_t>(row0) / static_cast<uint32_t>(group)), rem0 = row0 - i0 * group;
    // token of row row0 + r: rem0 + r is below 2^17, exact in binary32
    auto token_of = [&](int r) { return static_cast<int>((rem0 + r + 0.5f) * args.per_group); };
    const int i1 = i0 + uniform(token_of(min(R, rows - row0) - 1));
    const int kv_end = min(me.kv, args.room);
    const int first_pos = me.kv - me.m;
    const int end = min(max(first_pos + i1 + 1, 0), kv_end);
    int begin = 0;
    if (a.window > 0) begin = max(window_start(first_pos + i0, a.window), 0) & ~31;
    const int ntiles = end > begin ? (end - begin + 31) >> 5 : 0;
    // Nothing to see, maybe because the window begins past the table (a length is any 31-bit number):
    // no place is computed from there.
    if (ntiles == 0) begin = 0;
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
      const uint8_t* data = args.cache.data + static_cast<int64_t>(run.head) * 2 * page * D;
      const uint8_t* scales = args.cache.scales + static_cast<int64_t>(run.head) * 2 * (page / kBlock);
      const int32_t* table = a.table + run.request * a.table_stride;
      const int t_begin = begin + t_first * 32, t_end = min(begin + t_last * 32, end);

      // Where the keys of a half (16 tokens) start, and the scales of its block, one half a lane, from half
      // `base` of this part on; a valid place where there is nothing to see. The scales of the next
      // base are read a base ahead, their page ids two.
      constexpr int STEP = 48;  // halves between two bases: a round looks up to 15 ahead
      auto pages = [&](int h) {
        const int t = t_begin + (h + lane) * 16;
        return t < t_end ? table[t >> shift] : -1;
      };
      int base = 0;
      uint64_t k_at, seen;
      auto page_of = [&](int p) -> int64_t { return p >= 0 && p < num_pages ? p : 0; };
      auto scales_of = [&](int p, int h) -> uint32_t {
        const int off = (t_begin + (h + lane) * 16) & (page - 1);
        return *reinterpret_cast<const uint16_t*>(scales + page_of(p) * args.page_scales + off / kBlock * 2);
      };
      auto settle = [&](int p) {
        const int off = (t_begin + (base + lane) * 16) & (page - 1);
        k_at = reinterpret_cast<uint64_t>(data) + page_of(p) * args.page_bytes + off * D;
        seen = __ballot(p >= 0 && p < num_pages);
      };
      const int pages0 = pages(0);
      int pages_next = pages(STEP);
      uint32_t pair, pair_next;  // K's scale byte, then V's

      // This wave's rows.
      const int mine0 = row0 + wave * RW;
      int hi[NQ], lo[NQ];
      bf16x8 q[NQ][kSteps];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        // rows past the last repeat it
        const int r = min(wave * RW + n * 16 + c, rows - 1 - row0), i = i0 + token_of(r);
        const int pos = first_pos + i;
        hi[n] = min(pos + 1, kv_end);
        lo[n] = a.window > 0 ? window_start(pos, a.window) : 0;
        const uint16_t* x = static_cast<const uint16_t*>(a.q) + static_cast<int64_t>(me.q0 + i) * a.q_token +
                            static_cast<int64_t>(run.head * group + row0 + r - i * group) * a.q_head;
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
          q[n][k] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(x + step_at<D>(k, g)) ^ args.q_sign);
      }
      const int mine_end = mine0 < rows ? min(max(first_pos + i0 + token_of(min(wave * RW + RW, rows - row0) - 1) + 1, 0), kv_end) : 0;
      const int my_end = uniform(min(mine_end, t_end));
      // Units from here on need masks: the first row's end, the last row's window.
      const int i_first = i0 + token_of(min(wave * RW, rows - 1 - row0));
      const int whole_end = uniform(min(first_pos + i_first + 1, kv_end));
      const int whole_begin =
          uniform(a.window > 0 ? window_start(first_pos + i0 + token_of(min(wave * RW + RW, rows - row0) - 1), a.window) : 0);
      const int my_begin = uniform(a.window > 0 ? max(window_start(first_pos + i_first, a.window), 0) : 0);

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

      uint32_t keys[2][2][2 * kSteps];  // [this unit and the next, in turn][half]
      auto load_keys = [&](int h, uint32_t (*x)[2 * kSteps]) {
#pragma unroll
        for (int u = 0; u < 2; ++u) load_keys8<D>(lane_address(k_at, h + u - base), k_off, x[u]);
      };
      auto pair_of = [&](int h) { return static_cast<uint32_t>(lane_value(pair, h - base)); };
      u32x4 v[2][MINE];
      float v_scale[2];
      auto load_values = [&](int h) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const global_bytes kd = lane_address(k_at, h + u - base);
#pragma unroll
          for (int e = 0; e < MINE; ++e) v[u][e] = load_at<u32x4>(kd, v_off[e]);
          v_scale[u] = scale8_of(pair_of(h + u) >> 8);
        }
      };
      auto convert = [&](int buf) {
        uint32_t odd = 0;
#pragma unroll
        for (int e = 0; e < MINE; ++e)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t v0 = v[0][e][j], v1 = v[1][e][j];
            odd |= nan_codes(v0) | nan_codes(v1);
            values[buf][wave][4 * e + j][lane] = u32x4{codes8<0>(v0, v_scale[0]), codes8<1>(v0, v_scale[0]),
                                                       codes8<0>(v1, v_scale[1]), codes8<1>(v1, v_scale[1])};
          }
        const bool some = __any(odd != 0);
        if (lane == 0) reinterpret_cast<uint32_t*>(&any_nan[buf])[wave] = some;
      };

      const int halves = t_end > t_begin ? (t_end - t_begin + 15) >> 4 : 0;
      int buf = 0;
      settle(pages0);
      pair = scales_of(pages0, 0);
      pair_next = scales_of(pages_next, STEP);
      int pages_last = pages(2 * STEP);
      if (halves > 0) {
        load_values(my_unit * 2);
        load_keys(0, keys[0]);
        convert(0);
      }
      __syncthreads();
      for (int h0 = 0; h0 < halves; h0 += 2 * SUB) {
        const bool more = h0 + 2 * SUB < halves;
        const u32x4 some_nan = any_nan[buf];
        const bool round_nan = uniform(some_nan[0] | some_nan[1] | some_nan[2] | some_nan[3]) != 0;
        if (round_nan) {
          // NaN codes: added for the rows that see them and taken out, as masked ones times 0 would be NaN too.
#pragma unroll 1
          for (int sub = 0; sub < SUB; ++sub) {
            const int h = h0 + 2 * sub, t0 = t_begin + h * 16 + (thread_here() >> 4 & 3) * 4;
            const int both = static_cast<int>(seen >> (h - base)) & 3;
            bf16x8 visible[NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n)
              visible[n] = visible_of([&](int u, int i) {
                const int t = t0 + u * 16 + i;
                return t < hi[n] && t >= lo[n] && (both >> u & 1) != 0;
              });
#pragma unroll
            for (int j = 0; j < 4 * kSets; ++j) {
              const u32x4 x = values[buf][sub * SPLIT + j / OPS][j % OPS][lane];
#pragma unroll
              for (int n = 0; n < NQ; ++n) add_infinite(x, visible[n], acc[n][j >> 2][j & 3]);
              __builtin_amdgcn_sched_barrier(0);
            }
          }
          __syncthreads();
          take_out<DT_BF16, kAttnThreads>(reinterpret_cast<uint8_t*>(values[buf]), sizeof(values[buf]));
          __syncthreads();
        }
        if (more) load_values(h0 + 2 * SUB + my_unit * 2);
#pragma unroll 1
        for (int sub0 = 0; sub0 < SUB; sub0 += TURNS)
#pragma unroll
        for (int turn = 0; turn < TURNS; ++turn) {
          const int sub = sub0 + turn, h = h0 + 2 * sub;
          auto* now = keys[turn];
          load_keys(h + 2, keys[turn ^ 1]);
          const int t0 = t_begin + h * 16;
          if (t0 < my_end && t0 + 32 > my_begin) {
            const int both = static_cast<int>(seen >> (h - base)) & 3;  // the halves that have a page
            const bool masked = t0 + 32 > whole_end || t0 < whole_begin || both != 3;
            auto sees = [&](int n, int u, int i) {
              const int t = t0 + u * 16 + g * 4 + i;
              return t < hi[n] && t >= lo[n] && (both >> u & 1) != 0;
            };
            // Scores.
            __builtin_amdgcn_s_setprio(1);
            f32x4 s[NQ][2];
#pragma unroll
            for (int n = 0; n < NQ; ++n) s[n][0] = s[n][1] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float ks = scale8_of(pair_of(h + u) & 0xFFu);
#pragma unroll
              for (int i = 0; i < kSteps; ++i) {
                const bf16x8 kk = keys8(now[u], i, ks);
#pragma unroll
                for (int n = 0; n < NQ; ++n) s[n][u] = mfma(kk, q[n][i], s[n][u]);
              }
            }
            __builtin_amdgcn_s_setprio(0);
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
            bf16x8 vv[AHEAD];
            auto operand_of = [&](int j) {
              return __builtin_bit_cast(bf16x8, values[buf][sub * SPLIT + j / OPS][j % OPS][lane]);
            };
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) vv[j] = operand_of(j);
            __builtin_amdgcn_sched_barrier(0);
            // Probabilities.
            bf16x8 pr[NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              float top = s[n][0][0];
#pragma unroll
              for (int i = 1; i < 8; ++i) top = fmaxf(top, s[n][i >> 2][i & 3]);
              top *= args.scale_log2;
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
                x[i] = exp2_fast(fmaf(s[n][i >> 2][i & 3], args.scale_log2, -m[n]));
                l[n] += x[i];
              }
              split<1>(x, &pr[n]);
            }
            // Values.
#pragma unroll
            for (int j = 0; j < 4 * kSets; ++j) {
              const bf16x8 x = vv[j % AHEAD];
              if (j + AHEAD < 4 * kSets) vv[j % AHEAD] = operand_of(j + AHEAD);
#pragma unroll
              for (int n = 0; n < NQ; ++n) acc[n][j >> 2][j & 3] = mfma(x, pr[n], acc[n][j >> 2][j & 3]);
            }
          }
          if (TURNS == 1) {
#pragma unroll
            for (int i = 0; i < 2 * kSteps; ++i) keys[0][0][i] = keys[1][0][i], keys[0][1][i] = keys[1][1][i];
          }
        }
        __builtin_amdgcn_s_setprio(1);
        if (more) convert(buf ^ 1);
        __builtin_amdgcn_s_setprio(0);
        buf ^= 1;
        if (h0 + 2 * SUB - base == STEP) {
          base += STEP;
          settle(pages_next);
          pair = pair_next;
          pair_next = scales_of(pages_last, base + STEP);
          pages_next = pages_last;
          pages_last = pages(base + 2 * STEP);
        }
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
            for (int i = 0; i < 16; ++i) o[i] = acc[n][e][i & 3][i >> 2] * f;
            const int from = e * 64 + g * 16;
            if (parts > 1) {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                ar::st16<ar::kCoh>(part, (at * D + from + i) * 4,
                                   u32x4{__float_as_uint(o[i]), __float_as_uint(o[i + 1]), __float_as_uint(o[i + 2]),
                                         __float_as_uint(o[i + 3])});
            } else {
              u32x4* to = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + token * a.o_token + head * a.o_head + from);
#pragma unroll
              for (int i = 0; i < 16; i += 8)
                to[i / 8] = u32x4{ar::bf16x2_rne(o[i], o[i + 1]), ar::bf16x2_rne(o[i + 2], o[i + 3]),
                                  ar::bf16x2_rne(o[i + 4], o[i + 5]), ar::bf16x2_rne(o[i + 6], o[i + 7])};
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
          finish_row<DT_BF16>(a, me.q0 + i, head, seg, o0, o1, top, rl);
        };
        if (arrive(args.arrived + first_wg, parts, &last)) {
          const int real = min(R, rows - row0);
          if (parts == 2) join_few<D, R, 2, 4>(part, args.stats_at, first_wg, parts, real, finish);
          else if (parts <= 4) join_few<D, R, 4, 2>(part, args.stats_at, first_wg, parts, real, finish);
          else join_parts<D, R, 8>(part, args.stats_at, first_wg, parts, real, reinterpret_cast<float*>(values), finish);
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
          if (++run.request >= a.nreq) return;  // only if lengths change under the call
          me = wave_series(series_of<R>(args, run.request));
        } while (me.tiles == 0);
      }
    }
    span = uniform(me.below(run.tile + 1) - me.below(run.tile));
    __syncthreads();  // the next job uses the same LDS
  }
}

}  // namespace ard
