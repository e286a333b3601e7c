// Attention over the 4-bit paged cache for many query rows a request (prompt chunks), bfloat16.
//
// Mathematics as in ar_decode_attn_impl.h; the products are shared out the other way round: a
// workgroup's four waves hold 16 * NQ rows each and go through the same tokens together.
//
//   S^T = K Q^T   as there: a wave converts its own operands of K in registers, in the shadow of the
//                 products. (The scaled product takes K in its 4 bits, but a query only as e4m3
//                 values and drops what lies 2^-13 below the largest of eight products: 634
//                 against 640 us for two chunks of up to 2048 tokens against 12288, 32 heads, with
//                 elements below 2^-6 of the largest of their 32 cut.)
//   O^T += V^T P^T  V becomes bfloat16 (exactly) once a workgroup: each wave converts a quarter of a
//                 round's tokens into LDS in the order of the product's operand, for the next
//                 round while this one is computed. One barrier a round. P is one bfloat16 a
//                 value, as there; two (16 bits) took 874 us for the case above.
//
// Two waves share a SIMD. One of them multiplies while the other takes exponentials only if the products
// go first where both could issue: the scores and the conversions of V have a wave's higher priority
// (695 -> 640 us for the case above with the second operands read further ahead).
//
// Work. As there, equal runs of units for as many workgroups as the device holds; the units of a
// request's tiles grow with the tile (each sees the tokens before it), so they are summed as an
// arithmetic series. Consecutive runs lie on one XCD: they share keys and values in its L2.
#pragma once

#include "ar_decode_attn_impl.h"

namespace ard {

// A request as the split sees it: units of tile r (of one head) are below(r + 1) - below(r).
struct Series {
  int q0, m, kv, tiles;
  uint32_t first;     // units of tile 0
  double half_slope;  // half of what a tile has more than the one before
  __device__ uint32_t below(int r) const { return static_cast<uint32_t>(r * (first + (r - 1) * half_slope)); }
};

template <int R>
__device__ __forceinline__ Series series_of(const AttnArgs& args, int b) {
  const ar_kv4_attention_args& a = args.a;
  Series c = {0, 0, 0, 0, 1, 0.0};
  if (b < a.nreq) {
    const int at = a.q_start[b], to = a.q_start[b + 1];
    c.kv = max(a.kv_len[b], 0);
    c.q0 = min(max(at, 0), a.ntokens);
    c.m = max(min(to, a.ntokens) - c.q0, 0);
    c.tiles = static_cast<int>((static_cast<uint32_t>(c.m) * static_cast<uint32_t>(args.group) + R - 1) / R);
    const int end = min(c.kv, args.room);
    const int low = min(max(c.kv - c.m + min(args.tile_tokens, c.m), 0), end);
    auto units = [&](int seen) {
      return ((min(static_cast<uint32_t>(seen), args.most_seen) + args.unit - 1) >> args.unit_shift) + args.job_units;
    };
    c.first = units(low);
    if (c.tiles > 1) c.half_slope = static_cast<double>(units(end) - c.first) / (2 * (c.tiles - 1));
  }
  return c;
}

// The series that lane `l` holds.
__device__ __forceinline__ Series lane_series(const Series& c, int l) {
  const uint64_t slope = __builtin_bit_cast(uint64_t, c.half_slope);
  const uint32_t lo = lane_value(static_cast<uint32_t>(slope), l), hi = lane_value(static_cast<uint32_t>(slope >> 32), l);
  return {lane_value(c.q0, l), lane_value(c.m, l), lane_value(c.kv, l), lane_value(c.tiles, l),
          static_cast<uint32_t>(lane_value(c.first, l)),
          __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo)};
}

// As find_run, with a job's units in `span`.
template <int R>
__device__ __forceinline__ bool find_rows(const AttnArgs& args, int w, Run& run, Series& mine, int& span) {
  const int lane = threadIdx.x & 63, heads = args.cache.heads;
  uint32_t total = 0, longest = 0;
  Series c;
  uint32_t upto;
  for (int b = (args.a.nreq - 1) & ~63; b >= 0; b -= 64) {
    c = series_of<R>(args, b + lane);
    upto = wave_scan(c.below(c.tiles) * heads);
    longest = max(longest, wave_max(c.tiles > 0 ? c.below(c.tiles) - c.below(c.tiles - 1) : 0));
    total = __builtin_elementwise_add_sat(total, static_cast<uint32_t>(lane_value(upto, 63)));
  }
  if (total > 0x7FFFFFFFu) return false;  // request starts that overlap
  // Four units at least, a round of the workgroup; and parts of a job no shorter than makes reading
  // them back (one after the other, about 1.5 units each) as long as computing one.
  const int least = max((total + args.runs - 1) / args.runs,
                        static_cast<uint32_t>(uniform(static_cast<int>(sqrtf(1.5f * static_cast<float>(longest))))));
  run.per = max(4, least);
  if (static_cast<uint64_t>(w) * run.per >= total) return false;
  uint32_t from = w * run.per;
  run.left = min(run.per, static_cast<int>(total - from));
  int b = 0;
  while (__ballot(upto > from) == 0) {
    from -= lane_value(upto, 63);
    b += 64;
    if (b >= args.a.nreq) return false;  // only if lengths change under the call
    c = series_of<R>(args, b + lane);
    upto = wave_scan(c.below(c.tiles) * heads);
  }
  const int who = __builtin_ctzll(__ballot(upto > from));
  run.request = b + who;
  from -= who > 0 ? lane_value(upto, who - 1) : 0;
  // What the place was found by, not read again: head and tile stay inside it whatever changes.
  mine = lane_series(c, who);
  const uint32_t head_units = uniform(mine.below(mine.tiles));
  run.head = uniform(from / head_units);
  from -= run.head * head_units;
  // the tile: the root of the series, then to the whole number around it
  int r = 0;
  if (mine.tiles > 1) {
    const double h = mine.half_slope, f = mine.first - h;
    const double root = h > 0 ? (sqrt(f * f + 4 * h * from) - f) / (2 * h) : from / f;
    r = min(max(static_cast<int>(root), 0), mine.tiles - 1);
    while (r > 0 && mine.below(r) > from) --r;
    while (r + 1 < mine.tiles && mine.below(r + 1) <= from) ++r;
  }
  run.tile = uniform(r);
  run.at = uniform(from - mine.below(r));
  span = uniform(mine.below(r + 1) - mine.below(r));
  return true;
}

// A lane's share of 16 tokens' keys: a quarter of a row and the scales of the groups of 32 it lies in.
template <int D>
struct Keys16 {
  static constexpr int kDw = Tile32<D>::kDw, kKs = Tile32<D>::kKs;
  uint32_t k[kDw];
  uint32_t s[kKs];
};

template <int D, int NQ, int OCC>
__global__ __launch_bounds__(kAttnThreads, OCC) void kv4_attention_rows(AttnArgs args) {
  constexpr int RW = 16 * NQ, R = RW * kAttnWaves;
  constexpr int NC = D / 8, kSets = (NC + 15) / 16;
  constexpr int SUB = kAttnWaves / kSets;  // units of 32 tokens of a round
  constexpr int TURNS = kSets == 1 ? 2 : 1;  // units in the loop's body: with two, keys stay where they are
  typedef Keys16<D> Keys;
  constexpr int kDw = Keys::kDw, kKs = Keys::kKs;
  __shared__ u32x4 values[2][kAttnWaves][8][64];      // [buffer][unit, set][element][lane]
  __shared__ uint32_t nan_token[2][kAttnWaves][32];   // groups of 32 elements that are NaN
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
  const int k_bytes = page * (D / 2), s_bytes = page * (D / 32);
  const int num_pages = static_cast<int>(args.cache.num_pages);
  const int k_group = (g * kDw) >> 2;  // 32-group of a lane's first K dword
  const uint32_t k_off = c * (D / 2) + g * (D / 8);
  const int my_set = wave % kSets, my_unit = wave / kSets;
  const int chunk = min(my_set * 16 + c, NC - 1);
  const uint32_t v_off = k_bytes + g * (D * 2) + chunk * 16;
  const uint32_t vs_off = s_bytes + (chunk >> 2) * page + g * 4;
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
      const uint8_t* data = args.cache.data + static_cast<int64_t>(run.head) * 2 * k_bytes;
      const uint8_t* scales = args.cache.scales + static_cast<int64_t>(run.head) * 2 * s_bytes;
      const int32_t* table = a.table + run.request * a.table_stride;
      const int t_begin = begin + t_first * 32, t_end = min(begin + t_last * 32, end);

      // Where the keys of a half (16 tokens) and its scales start, one half a lane, from half
      // `base` of this part on; a valid place where there is nothing to see. Wide address
      // arithmetic for every half in turn was a third of the loop's instructions.
      constexpr int STEP = 48;  // halves between two bases: a round looks up to 15 ahead
      auto pages = [&](int h) {
        const int t = t_begin + (h + lane) * 16;
        return t < t_end ? table[t >> shift] : -1;
      };
      int base = 0;
      uint64_t k_at, s_at, seen;
      auto settle = [&](int p) {
        const bool some = p >= 0 && p < num_pages;
        const int64_t at = some ? p : 0;
        const int off = (t_begin + (base + lane) * 16) & (page - 1);
        k_at = reinterpret_cast<uint64_t>(data) + at * args.page_bytes + off * (D / 2);
        s_at = reinterpret_cast<uint64_t>(scales) + at * args.page_scales + off;
        seen = __ballot(some);
      };
      const int pages0 = pages(0);
      int pages_next = pages(STEP);

      // This wave's rows.
      const int mine0 = row0 + wave * RW;
      int hi[NQ], lo[NQ];
      bf16x8 q[NQ][kDw];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        // rows past the last repeat it
        const int r = min(wave * RW + n * 16 + c, rows - 1 - row0), i = i0 + token_of(r);
        const int pos = first_pos + i;
        hi[n] = min(pos + 1, kv_end);
        lo[n] = a.window > 0 ? window_start(pos, a.window) : 0;
        const uint16_t* x = static_cast<const uint16_t*>(a.q) + static_cast<int64_t>(me.q0 + i) * a.q_token +
                            static_cast<int64_t>(run.head * group + row0 + r - i * group) * a.q_head + g * (D / 4);
#pragma unroll
        for (int k = 0; k < kDw; ++k)
          q[n][k] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(x + k * 8) ^ args.q_sign);
      }
      const int mine_end = mine0 < rows ? min(max(first_pos + i0 + token_of(min(wave * RW + RW, rows - row0) - 1) + 1, 0), kv_end) : 0;
      const int my_end = uniform(min(mine_end, t_end));
      // Units from here on need masks: the first row's end, the last row's window.
      const int i_first = i0 + token_of(min(wave * RW, rows - 1 - row0));
      const int whole_end = uniform(min(first_pos + i_first + 1, kv_end));
      const int whole_begin =
          uniform(a.window > 0 ? window_start(first_pos + i0 + token_of(min(wave * RW + RW, rows - row0) - 1), a.window) : 0);
      const int my_begin = uniform(a.window > 0 ? max(window_start(first_pos + i_first, a.window), 0) : 0);

      f32x4 acc[NQ][kSets][8];
      float m[NQ], l[NQ];
      int nan_groups[NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        m[n] = kLowest, l[n] = 0.0f, nan_groups[n] = 0;
#pragma unroll
        for (int e = 0; e < kSets; ++e)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[n][e][j] = f32x4{0, 0, 0, 0};
      }

      auto load_keys = [&](int h, Keys* x) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const global_bytes kd = lane_address(k_at, h + u - base), sd = lane_address(s_at, h + u - base);
          load_dwords<kDw>(kd, k_off, x[u].k);
#pragma unroll
          for (int i = 0; i < kKs; ++i) x[u].s[i] = load_at<uint8_t>(sd, min(k_group + i, D / 32 - 1) * page + c);
        }
      };
      u32x4 v[2];
      uint32_t vs[2];
      auto load_values = [&](int h) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const global_bytes kd = lane_address(k_at, h + u - base), sd = lane_address(s_at, h + u - base);
          v[u] = load_at<u32x4>(kd, v_off);
          vs[u] = load_at<uint32_t>(sd, vs_off);
        }
      };
      auto convert = [&](int buf) {
        uint32_t bad[2] = {nan_bytes(vs[0]), nan_bytes(vs[1])};
        const bool some = __any((bad[0] | bad[1]) != 0);
        if (lane == 0) reinterpret_cast<uint32_t*>(&any_nan[buf])[wave] = some;
        if (lane < 32) nan_token[buf][wave][lane] = 0;
        if (some) {  // read as finite; the rows that see them are noted from nan_token
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if ((c & 3) == 0 && my_set * 16 + c < NC)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (bad[u] >> (8 * i + 7) & 1) atomicOr(&nan_token[buf][wave][u * 16 + g * 4 + i], 1u << (chunk >> 2));
            bad[u] |= bad[u] >> 1, bad[u] |= bad[u] >> 2, bad[u] |= bad[u] >> 4;
            vs[u] &= ~bad[u];
          }
        }
        float sc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) sc[i] = __uint_as_float((vs[i >> 2] >> (8 * (i & 3)) & 0xFFu) << 23);
#define ARD_PAIR(B)                                                                               \
  {                                                                                               \
    uint32_t x[8];                                                                                \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) x[i] = codes<B>(v[i >> 2][i & 3], sc[i]);       \
    values[buf][wave][2 * B][lane] =                                                              \
        u32x4{pair_lo(x[0], x[1]), pair_lo(x[2], x[3]), pair_lo(x[4], x[5]), pair_lo(x[6], x[7])}; \
    values[buf][wave][2 * B + 1][lane] =                                                          \
        u32x4{pair_hi(x[0], x[1]), pair_hi(x[2], x[3]), pair_hi(x[4], x[5]), pair_hi(x[6], x[7])}; \
  }
        ARD_PAIR(0) ARD_PAIR(1) ARD_PAIR(2) ARD_PAIR(3)
#undef ARD_PAIR
      };

      const int halves = t_end > t_begin ? (t_end - t_begin + 15) >> 4 : 0;
      int buf = 0;
      Keys keys[2][2];  // of this unit and the next, in turn
      settle(pages0);
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
        if (more) load_values(h0 + 2 * SUB + my_unit * 2);
#pragma unroll 1
        for (int sub0 = 0; sub0 < SUB; sub0 += TURNS)
#pragma unroll
        for (int turn = 0; turn < TURNS; ++turn) {
          const int sub = sub0 + turn, h = h0 + 2 * sub;
          const Keys* now = keys[turn];
          load_keys(h + 2, keys[turn ^ 1]);
          const int t0 = t_begin + h * 16;
          if (t0 < my_end && t0 + 32 > my_begin) {
            // Scores.
            __builtin_amdgcn_s_setprio(1);
            f32x4 s[NQ][2];
#pragma unroll
            for (int n = 0; n < NQ; ++n) s[n][0] = s[n][1] = f32x4{0, 0, 0, 0};
            float sc[2][kKs];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int i = 0; i < kKs; ++i) sc[u][i] = scale_of(now[u].s[i]);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int i = 0; i < kDw; ++i) {
                float x = sc[u][0];
                if (kKs > 1) x = ((g * kDw + i) >> 2) == k_group ? sc[u][0] : sc[u][kKs - 1];
                const uint32_t w = now[u].k[i];
                const bf16x8 kk = operand(codes<0>(w, x), codes<1>(w, x), codes<2>(w, x), codes<3>(w, x));
#pragma unroll
                for (int n = 0; n < NQ; ++n) s[n][u] = mfma(kk, q[n][i], s[n][u]);
              }
            __builtin_amdgcn_s_setprio(0);
            const int both = static_cast<int>(seen >> (h - base)) & 3;  // the halves that have a page
            if (t0 + 32 > whole_end || t0 < whole_begin || both != 3) {
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
            // The first operands of the second product, under way with the probabilities.
            constexpr int AHEAD = 8;
            bf16x8 vv[AHEAD];
            auto operand_of = [&](int j) {
              return __builtin_bit_cast(bf16x8, values[buf][sub * kSets + (j >> 3)][j & 7][lane]);
            };
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) vv[j] = operand_of(j);
            __builtin_amdgcn_sched_barrier(0);
            if (round_nan) {
#pragma unroll 1
              for (int x = 0; x < 32 * kSets; ++x) {
                const uint32_t groups = nan_token[buf][sub * kSets + (x >> 5)][x & 31];
                const int t = t0 + (x & 31);
                if (groups == 0 || (both >> (x >> 4 & 1) & 1) == 0) continue;
#pragma unroll
                for (int n = 0; n < NQ; ++n)
                  if (t < hi[n] && t >= lo[n]) nan_groups[n] |= groups;
              }
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
                  for (int j = 0; j < 8; ++j) acc[n][e][j] *= f;
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
            for (int j = 0; j < 8 * kSets; ++j) {
              const bf16x8 x = vv[j % AHEAD];
              if (j + AHEAD < 8 * kSets) vv[j % AHEAD] = operand_of(j + AHEAD);
#pragma unroll
              for (int n = 0; n < NQ; ++n) acc[n][j >> 3][j & 7] = mfma(x, pr[n], acc[n][j >> 3][j & 7]);
            }
          }
          if (TURNS == 1) keys[0][0] = keys[1][0], keys[0][1] = keys[1][1];
        }
        __builtin_amdgcn_s_setprio(1);
        if (more) convert(buf ^ 1);
        __builtin_amdgcn_s_setprio(0);
        buf ^= 1;
        if (h0 + 2 * SUB - base == STEP) {
          base += STEP;
          settle(pages_next);
          pages_next = pages(base + STEP);
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
            const bool nan = nan_groups[n] >> (e * 4 + g) & 1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int to_chunk = e * 16 + g * 4 + k;
              if (to_chunk >= NC) continue;
              float o[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) o[j] = nan ? __uint_as_float(0x7FC00000u) : acc[n][e][j][k] * f;
              if (parts > 1) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  ar::st16<ar::kCoh>(part, (at * D + to_chunk * 8 + 4 * j) * 4,
                                     u32x4{__float_as_uint(o[4 * j]), __float_as_uint(o[4 * j + 1]),
                                           __float_as_uint(o[4 * j + 2]), __float_as_uint(o[4 * j + 3])});
              } else {
                *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + token * a.o_token + head * a.o_head + to_chunk * 8) =
                    u32x4{ar::bf16x2_rne(o[0], o[1]), ar::bf16x2_rne(o[2], o[3]), ar::bf16x2_rne(o[4], o[5]),
                          ar::bf16x2_rne(o[6], o[7])};
              }
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
