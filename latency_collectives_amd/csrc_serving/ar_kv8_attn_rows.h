// Attention over the 8-bit paged cache for many query rows a request (prompt chunks), bfloat16.
//
// Mathematics, split of the work and joins as in csrc_decode/ar_decode_attn_rows.h; operands as in
// ar_kv8_attn.h. A workgroup's waves hold 16 * NQ rows each and go through the same tokens together. Keys and values
// become bfloat16 (exactly) once a workgroup: each wave converts its share of a round into LDS in the order of the
// products' operands, for the next round while this one is computed, from codes that it loaded before. One
// barrier a round. With each wave converting the keys it multiplies by in its registers, two waves a SIMD was what fitted:
// 657 us for two chunks of up to 2048 tokens against 12288, 32 heads of 128 on 8; so 571.
#pragma once

#include "../csrc_decode/ar_decode_attn_rows.h"
#include "ar_kv8_attn.h"

namespace ard {

template <int D, int NQ, int WAVES, int SUB, int OCC>
__global__ __launch_bounds__(64 * WAVES, OCC) void kv8_attention_rows(AttnArgs given) {
  constexpr int RW = 16 * NQ, R = RW * WAVES, THREADS = 64 * WAVES;
  constexpr int kSteps = D / 32, kSets = (D + 63) / 64;
  // A wave's items of a round: one set of a unit's values, or two steps of its keys, of both its halves.
  constexpr int kItems = SUB * 2 * kSets, kMine = (kItems + WAVES - 1) / WAVES;
  static_assert((kSteps + 1) / 2 == kSets && 48 % (2 * SUB) == 0 && SUB <= 8);
  struct Round {
    u32x4 keys[SUB][2][kSteps][64];   // [unit][half][step][lane]
    u32x4 values[SUB][kSets][4][64];  // [unit][set][operand][lane]
  };
  struct Lds {
    Round round[2];
    uint32_t odd[2][WAVES];
  };
  __shared__ Lds lds;
  __shared__ int last;

  const AttnArgs& args = given;
  // consecutive runs on one XCD: workgroups go to the eight in turn
  const int w = (blockIdx.x & 7) * (args.runs >> 3) + (blockIdx.x >> 3);
  Run run;
  Series me;
  int span;
  if (!find_rows<R>(args, w, run, me, span)) return;
  const int wave = uniform(threadIdx.x >> 6);
  const int group = args.group, shift = args.cache.page_shift;
  const int page = 1 << shift;
  const int num_pages = static_cast<int>(args.cache.num_pages);
  auto lane_here = [] { return thread_here() & 63; };
  // Where a lane's elements of item x of a unit lie from a half's first key on.
  auto item_off = [&](int x) -> uint32_t {
    const int c = lane_here() & 15, g = lane_here() >> 4;
    return x < kSets ? c * D + step_at<D>(2 * x, g)
                     // lanes beyond the row repeat its last elements
                     : page * D + g * (4 * D) + min((x - kSets) * 64 + c * 4, D - 4) * 4;
  };
  constexpr uint32_t kValues = sizeof(lds.round[0].keys);
  const uint32_t lds_base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((ARD_LDS Lds*)&lds)) + lane_here() * 16;

  for (;;) {
    const AttnArgs& args = args_here<AttnArgs>();
    const ar_kv4_attention_args& a = args.a;
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
      // base are read half a base ahead, their page ids a base.
      constexpr int STEP = 48;  // halves between two bases: a round looks up to 15 ahead
      constexpr int HALF = 24 / (2 * SUB) * (2 * SUB);
      auto pages = [&](int h) {
        const int t = t_begin + (h + lane_here()) * 16;
        return t < t_end ? table[t >> shift] : -1;
      };
      int base = 0;
      uint64_t k_at, seen;
      auto page_of = [&](int p) -> int64_t { return p >= 0 && p < num_pages ? p : 0; };
      auto scales_of = [&](int p, int h) -> uint32_t {
        const int off = (t_begin + (h + lane_here()) * 16) & (page - 1);
        return *reinterpret_cast<const uint16_t*>(scales + page_of(p) * args.page_scales + off / kBlock * 2);
      };
      auto settle = [&](int p) {
        const int off = (t_begin + (base + lane_here()) * 16) & (page - 1);
        k_at = reinterpret_cast<uint64_t>(data) + page_of(p) * args.page_bytes + off * D;
        seen = __ballot(p >= 0 && p < num_pages);
      };
      const int pages0 = pages(0);
      int pages_next = pages(STEP);
      uint32_t pair, pair_next = 0;  // K's scale byte, then V's

      // This wave's rows.
      const int mine0 = row0 + wave * RW;
      int pos[NQ];
      bf16x8 q[NQ][kSteps];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        // rows past the last repeat it
        const int c = thread_here() & 15, g = thread_here() >> 4 & 3;
        const int r = min(wave * RW + n * 16 + c, rows - 1 - row0), i = i0 + token_of(r);
        pos[n] = first_pos + i;
        const uint16_t* x = static_cast<const uint16_t*>(a.q) + static_cast<int64_t>(me.q0 + i) * a.q_token +
                            static_cast<int64_t>(run.head * group + row0 + r - i * group) * a.q_head;
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
          q[n][k] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(x + step_at<D>(k, g)) ^ args.q_sign);
      }
      auto sees = [&](int n, int t) {
        return t <= pos[n] && t < kv_end && (a.window <= 0 || t >= window_start(pos[n], a.window));
      };
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
          for (int j = 0; j < 4; ++j) acc[n][e][j] = zeros_here();
      }

      auto pair_of = [&](int h) { return static_cast<uint32_t>(lane_value(pair, h - base)); };
      u32x4 raw[kMine][2];  // [half]
      float scale[kMine][2];
      auto item = [&](int k) { return wave + k * WAVES; };
      auto load = [&](int h0) {
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
          if (kItems % WAVES != 0 && item(k) >= kItems) continue;
          const int x = item(k) % (2 * kSets), h = h0 + item(k) / (2 * kSets) * 2;
          const uint32_t off = item_off(x);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const global_bytes kd = lane_address(k_at, h + u - base);
            if (D % 64 != 0 && x < kSets) {
              const u32x2 y = load_at<u32x2>(kd, off), z = load_at<u32x2>(kd, off + (2 * x + 1 < kSteps ? 32 : 0));
              raw[k][u] = u32x4{y.x, y.y, z.x, z.y};
            } else {
              raw[k][u] = load_at<u32x4>(kd, off);
            }
            scale[k][u] = scale8_of(pair_of(h + u) >> (x < kSets ? 0 : 8) & 0xFFu);
          }
        }
      };
      auto put = [](uint32_t to, u32x4 x) { *reinterpret_cast<ARD_LDS u32x4*>(to) = x; };
      auto convert = [&](int buf) {
        uint32_t to = lds_base + buf * static_cast<uint32_t>(sizeof(Round));
        asm("" : "+v"(to));
        uint32_t odd = 0;
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
          if (kItems % WAVES != 0 && item(k) >= kItems) continue;
          const int x = item(k) % (2 * kSets), unit = item(k) / (2 * kSets);
          auto codes = [&](int u, int i) { return codes8<0>(raw[k][u][i], scale[k][u]); };
          auto codes_high = [&](int u, int i) { return codes8<1>(raw[k][u][i], scale[k][u]); };
          if (x < kSets) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int s = 0; s < 2; ++s)
                if (kSteps % 2 == 0 || 2 * x + s < kSteps)
                  put(to + (((unit * 2 + u) * kSteps) + 2 * x + s) * 1024,
                      u32x4{codes(u, 2 * s), codes_high(u, 2 * s), codes(u, 2 * s + 1), codes_high(u, 2 * s + 1)});
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              odd |= nan_codes(raw[k][0][j]) | nan_codes(raw[k][1][j]);
              put(to + kValues + ((unit * kSets + x - kSets) * 4 + j) * 1024,
                  u32x4{codes(0, j), codes_high(0, j), codes(1, j), codes_high(1, j)});
            }
          }
        }
        const bool some = __any(odd != 0);
        if (lane_here() == 0) lds.odd[buf][wave] = some;
      };

      const int halves = t_end > t_begin ? (t_end - t_begin + 15) >> 4 : 0;
      int buf = 0;
      settle(pages0);
      pair = scales_of(pages0, 0);
      if (halves > 0) {
        load(0);
        convert(0);
      }
      __syncthreads();
#pragma unroll 1
      for (int h0 = 0; h0 < halves; h0 += 2 * SUB) {
        const bool more = h0 + 2 * SUB < halves;
        uint32_t odd = 0;
#pragma unroll
        for (int x = 0; x < WAVES; ++x) odd |= lds.odd[buf][x];
        if (uniform(odd) != 0) {
          // NaN codes: added for the rows that see them and taken out, as masked ones times 0 would be NaN too.
#pragma unroll 1
          for (int sub = 0; sub < SUB; ++sub) {
            const int h = h0 + 2 * sub, t0 = t_begin + h * 16 + (thread_here() >> 4 & 3) * 4;
            const int both = static_cast<int>(seen >> (h - base)) & 3;
            bf16x8 visible[NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n)
              visible[n] = visible_of([&](int u, int i) { return sees(n, t0 + u * 16 + i) && (both >> u & 1) != 0; });
#pragma unroll
            for (int j = 0; j < 4 * kSets; ++j) {
              const u32x4 x = lds.round[buf].values[sub][j >> 2][j & 3][lane_here()];
#pragma unroll
              for (int n = 0; n < NQ; ++n) add_infinite(x, visible[n], acc[n][j >> 2][j & 3]);
              __builtin_amdgcn_sched_barrier(0);
            }
          }
          __syncthreads();
          take_out<DT_BF16, THREADS>(reinterpret_cast<uint8_t*>(lds.round[buf].values), sizeof(lds.round[buf].values));
          __syncthreads();
        }
        if (more) load(h0 + 2 * SUB);
        uint32_t from = lds_base + buf * static_cast<uint32_t>(sizeof(Round));
        asm("" : "+v"(from));  // operands are offsets from it
        // The first keys of a unit are read before the unit before it ends.
        constexpr int EARLY = 2 * kSteps < 6 ? 2 * kSteps : 6;
        u32x4 kf[EARLY];
        auto read_key = [&](int sub, int i) { return lds_at<u32x4>(from + ((sub * 2 + (i & 1)) * kSteps + (i >> 1)) * 1024); };
        auto read_first = [&](int sub) {
#pragma unroll
          for (int i = 0; i < EARLY; ++i) kf[i] = read_key(sub, i);
        };
        read_first(0);
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub) {
          const int h = h0 + 2 * sub, t0 = t_begin + h * 16;
          if (t0 >= my_end || t0 + 32 <= my_begin) {
            if (sub + 1 < SUB) read_first(sub + 1);
          } else {
            const int both = static_cast<int>(seen >> (h - base)) & 3;  // the halves that have a page
            const bool masked = t0 + 32 > whole_end || t0 < whole_begin || both != 3;
            // Scores.
            __builtin_amdgcn_s_setprio(1);
            f32x4 s[NQ][2];
#pragma unroll
            for (int n = 0; n < NQ; ++n) s[n][0] = s[n][1] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const bf16x8 kk = __builtin_bit_cast(bf16x8, i * 2 + u < EARLY ? kf[i * 2 + u] : read_key(sub, i * 2 + u));
#pragma unroll
                for (int n = 0; n < NQ; ++n) s[n][u] = mfma(kk, q[n][i], s[n][u]);
              }
            __builtin_amdgcn_s_setprio(0);
            // The first operands of the second product, under way with the probabilities.
            constexpr int AHEAD = 4;
            bf16x8 vv[4 * kSets];
            auto read_value = [&](int j) { vv[j] = __builtin_bit_cast(bf16x8, lds_at<u32x4>(from + kValues + (sub * kSets * 4 + j) * 1024)); };
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) read_value(j);
            __builtin_amdgcn_sched_barrier(0);
            if (masked) {
              const int first = t0 + (thread_here() >> 4 & 3) * 4;
#pragma unroll
              for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    if (!sees(n, first + u * 16 + i) || (both >> u & 1) == 0) s[n][u][i] = -INFINITY;
            }
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
              if (j >= AHEAD) read_value(j);
              if (j == 2 * kSets && sub + 1 < SUB) read_first(sub + 1);
#pragma unroll
              for (int n = 0; n < NQ; ++n) acc[n][j >> 2][j & 3] = mfma(vv[j], pr[n], acc[n][j >> 2][j & 3]);
            }
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
          pages_next = pages(base + STEP);
        } else if (h0 + 2 * SUB - base == HALF) {
          pair_next = scales_of(pages_next, base + STEP);
        }
        __syncthreads();
      }

      // This wave's rows are its own: out, or into the workspace. (Places computed anew: kept from job to job they
      // would take the loop's registers.)
      const AttnArgs& args = args_here<AttnArgs>();
      const ar_kv4_attention_args& a = args.a;
      const ar::rsrc_t part = ar::make_rsrc(args.part, args.part_bytes);
      const int here = thread_here() & 63, c = here & 15, g = here >> 4;
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
              a.lse[token * a.q_heads + head] = l[n] == 0.0f ? -INFINITY : (m[n] + __builtin_amdgcn_logf(l[n])) * 0.6931471805599453f;
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
          if (parts == 2) join_few<D, R, 2, 4, true, THREADS>(part, args.stats_at, first_wg, parts, real, finish);
          else if (parts <= 4) join_few<D, R, 4, 2, true, THREADS>(part, args.stats_at, first_wg, parts, real, finish);
          else join_parts<D, R, 8, true, THREADS>(part, args.stats_at, first_wg, parts, real, reinterpret_cast<float*>(&lds), finish);
        }
      }
    }
    if (run.left <= 0) return;
    // The next job of the run.
    {
    const AttnArgs& args = args_here<AttnArgs>();
    run.at = 0;
    if (++run.tile == me.tiles) {
      run.tile = 0;
      if (++run.head == args.cache.heads) {
        run.head = 0;
        do {
          if (++run.request >= args.a.nreq) return;  // only if lengths change under the call
          me = wave_series(series_of<R>(args, run.request));
        } while (me.tiles == 0);
      }
    }
    }
    span = uniform(me.below(run.tile + 1) - me.below(run.tile));
    __syncthreads();  // the next job uses the same LDS
  }
}

}  // namespace ard
