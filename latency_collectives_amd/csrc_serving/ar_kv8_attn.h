// Attention over the 8-bit paged cache (gfx950): tiles of 16 or 32 rows, waves on different tokens.
//
// Mathematics, split of the work and joins are those of the attention over the 4-bit cache
// (csrc_decode/ar_decode_attn_impl.h). What differs is how tokens become operands:
//
//   S^T [32 tokens x 16 rows] = K Q^T   lane (c, g) reads sixteen bytes of token c's row at 16 g of
//                 every 64: two steps of the product. A step's elements are the same ones of the
//                 query, so their order does not matter.
//   O^T [D x 16 rows] += V^T P^T   a lane reads four elements of four tokens in one load; a word is one
//                 element of four tokens, which two conversions make half an operand: no permutes.
//
// Probabilities of bfloat16 calls are one bfloat16, as there; of binary32 calls three, as the query is.
//
// Two codes are one conversion, scaled by their block's power of two, exactly; a block of 16 tokens is
// half a tile, so its scales are scalars of the wave.
//
// Bound by the cache's bytes: 64 requests of up to 8192 tokens, 8 kv heads of 128 (536 MB), 102 us, 5.2 TB/s; head of 64 46 us, of 256
// 189; binary32 108; one request of 2000 tokens, one kv head, 8.1, bound by latency.
#pragma once

#include "ar_kv8.h"

namespace ard {

template <int D>
struct Tile8 {  // a lane's share of 32 tokens, as loaded
  static constexpr int kSteps = D / 32;          // of the first product
  static constexpr int kSets = (D + 63) / 64;    // loads of a value's elements, four products each
  uint32_t k[2][2 * kSteps];
  u32x4 v[2][kSets];
};

// Where a lane's elements of step s begin in a row.
template <int D>
__device__ __forceinline__ constexpr int step_at(int s, int g) {
  return D % 64 == 0 ? (s >> 1) * 64 + g * 16 + (s & 1) * 8 : s * 32 + g * 8;
}
template <int D>
__device__ __forceinline__ void load_keys8(global_bytes p, uint32_t off, uint32_t* k) {
  constexpr int kSteps = D / 32;
  if (D % 64 == 0) {
#pragma unroll
    for (int j = 0; j < kSteps / 2; ++j) {
      const u32x4 x = load_at<u32x4>(p, off + 64 * j);
#pragma unroll
      for (int i = 0; i < 4; ++i) k[4 * j + i] = x[i];
    }
  } else {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const u32x2 x = load_at<u32x2>(p, off + 32 * s);
      k[2 * s] = x.x, k[2 * s + 1] = x.y;
    }
  }
}
// One step's operand of the keys.
__device__ __forceinline__ bf16x8 keys8(const uint32_t* k, int s, float scale) {
  return operand(codes8<0>(k[2 * s], scale), codes8<1>(k[2 * s], scale), codes8<0>(k[2 * s + 1], scale),
                 codes8<1>(k[2 * s + 1], scale));
}

template <int DT, int D, int NQ, int OCC>
__global__ __launch_bounds__(kAttnThreads, OCC) void kv8_attention(AttnArgs args) {
  constexpr int R = 16 * NQ;
  constexpr int PARTS = DT == DT_BF16 ? 1 : 3;
  constexpr int NC = D / 8;
  typedef Tile8<D> Tile;
  constexpr int kSteps = Tile::kSteps, kSets = Tile::kSets;
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
  const int page = 1 << shift;
  const int num_pages = static_cast<int>(args.cache.num_pages);
  // Per-lane offsets within 16 tokens' keys and values.
  const uint32_t k_off = c * D + step_at<D>(0, g);
  uint32_t v_off[kSets];
#pragma unroll
  for (int e = 0; e < kSets; ++e)  // lanes beyond the row repeat its last elements
    v_off[e] = page * D + g * (4 * D) + min(e * 64 + c * 4, D - 4) * 4;

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
      const uint8_t* data = args.cache.data + static_cast<int64_t>(run.head) * 2 * page * D;
      const uint8_t* scales = args.cache.scales + static_cast<int64_t>(run.head) * 2 * (page / kBlock);
      const int32_t* table = a.table + run.request * a.table_stride;

      // Where the keys of this wave's next 32 tiles start, and the scales of their blocks: lane 2 k + u has
      // the u-th half of the k-th, a valid place where there is nothing to see.
      auto pages = [&](int tile) {
        const int mine = tile + (lane >> 1) * kAttnWaves, t = begin + mine * 32 + (lane & 1) * 16;
        return mine < t_last && t < end ? table[t >> shift] : -1;
      };
      uint64_t k_at, seen;
      uint32_t pair = 0;  // K's scale byte, then V's
      auto settle = [&](int p) {
        const bool some = p >= 0 && p < num_pages;
        const int64_t at = some ? p : 0;
        const int off = (begin + (t_first + wave) * 32 + (lane & 1) * 16 + (lane >> 1) * (kAttnWaves * 32)) & (page - 1);
        k_at = reinterpret_cast<uint64_t>(data) + at * args.page_bytes + off * D;
        pair = *reinterpret_cast<const uint16_t*>(scales + at * args.page_scales + off / kBlock * 2);
        seen = __ballot(some);
      };
      int ids = pages(t_first + wave);  // under way with the queries

      int hi[NQ], lo[NQ];
      bf16x8 q[NQ][PARTS][kSteps];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const int row = row0 + n * 16 + c;
        const bool real = row < rows;  // others repeat the last row, with nothing to see
        const int r = min(n * 16 + c, rows - 1 - row0), i = i0 + token_of(r);
        const int pos = first_pos + i;
        hi[n] = real ? min(pos + 1, kv_end) : 0;
        lo[n] = a.window > 0 ? window_start(pos, a.window) : 0;
        const int64_t at = static_cast<int64_t>(me.q0 + i) * a.q_token +
                           static_cast<int64_t>(run.head * group + row0 + r - i * group) * a.q_head;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const int64_t from = at + step_at<D>(s, g);
          if (DT == DT_BF16) {
            const u32x4 x = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.q) + from);
            q[n][0][s] = __builtin_bit_cast(bf16x8, x);
          } else {
            float x[8];
            const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(a.q) + from);
            const f32x4 v0 = p[0], v1 = p[1];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = v0[j], x[4 + j] = v1[j];
            bf16x8 y[PARTS];
            split<PARTS>(x, y);
#pragma unroll
            for (int p = 0; p < PARTS; ++p) q[n][p][s] = y[p];
          }
        }
      }
      // Tiles from here on need masks: the first row's end, the last row's window.
      const int whole_end = min(first_pos + i0 + 1, kv_end);
      const int whole_begin = a.window > 0 ? window_start(first_pos + i1, a.window) : 0;

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

      auto load = [&](int k, Tile& x) {
#pragma unroll
        for (int u = 0; u < 2; ++u) load_keys8<D>(lane_address(k_at, 2 * k + u), k_off, x.k[u]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const global_bytes kd = lane_address(k_at, 2 * k + u);
#pragma unroll
          for (int e = 0; e < kSets; ++e) x.v[u][e] = load_at<u32x4>(kd, v_off[e]);
        }
      };

      // The first round only loads: one copy of this code.
      Tile now, next;
      int tile = t_first + wave - kAttnWaves, turn = 0;
      int both = 0, both_next;  // the halves that have a page
      for (; tile < t_last; tile += kAttnWaves) {
        const int k_now = (turn + 31) & 31;
        const uint32_t pair0 = lane_value(pair, 2 * k_now), pair1 = lane_value(pair, 2 * k_now + 1);
        if ((turn & 31) == 0) {
          settle(ids);
          ids = pages(tile + 33 * kAttnWaves);
        }
        both_next = static_cast<int>(seen >> (2 * (turn & 31))) & 3;
        load(turn++ & 31, next);
        if (tile >= t_first) {
          const int t0 = begin + tile * 32;
          const float ks[2] = {scale8_of(pair0 & 0xFFu), scale8_of(pair1 & 0xFFu)};
          const float vs[2] = {scale8_of(pair0 >> 8), scale8_of(pair1 >> 8)};
          const bool masked = t0 + 32 > whole_end || t0 < whole_begin || both != 3;
          auto sees = [&](int n, int u, int i) {
            const int t = t0 + u * 16 + g * 4 + i;
            return t < hi[n] && t >= lo[n] && (both >> u & 1) != 0;
          };
          if (masked) {  // values that are NaN, of tokens that only some rows see
            uint32_t odd = 0;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int e = 0; e < kSets; ++e)
#pragma unroll
                for (int j = 0; j < 4; ++j) odd |= nan_codes(now.v[u][e][j]);
            if (__any(odd != 0)) {
              bf16x8 visible[NQ];
#pragma unroll
              for (int n = 0; n < NQ; ++n) visible[n] = visible_of([&](int u, int i) { return sees(n, u, i); });
#pragma unroll
              for (int e = 0; e < kSets; ++e)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  u32x4 x;
#pragma unroll
                  for (int u = 0; u < 2; ++u) {
                    const uint32_t code = now.v[u][e][j];
                    x[2 * u] = codes8<0>(code, vs[u]), x[2 * u + 1] = codes8<1>(code, vs[u]);
                    uint32_t bad = nan_codes(code);
                    bad |= bad >> 1, bad |= bad >> 2, bad |= bad >> 4;
                    now.v[u][e][j] = code & ~bad;
                  }
#pragma unroll
                  for (int n = 0; n < NQ; ++n) add_infinite(x, visible[n], acc[n][e][j]);
                  __builtin_amdgcn_sched_barrier(0);
                }
            }
          }
          // Scores.
          f32x4 s[NQ][2];
#pragma unroll
          for (int n = 0; n < NQ; ++n) s[n][0] = s[n][1] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
              const bf16x8 kk = keys8(now.k[u], i, ks[u]);
#pragma unroll
              for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int p = 0; p < PARTS; ++p) s[n][u] = mfma(kk, q[n][p][i], s[n][u]);
            }
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
                for (int j = 0; j < 4; ++j) acc[n][e][j] *= f;
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
          for (int e = 0; e < kSets; ++e)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t v0 = now.v[0][e][j], v1 = now.v[1][e][j];
              const bf16x8 vv = operand(codes8<0>(v0, vs[0]), codes8<1>(v0, vs[0]), codes8<0>(v1, vs[1]), codes8<1>(v1, vs[1]));
#pragma unroll
              for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int p = 0; p < PARTS; ++p) acc[n][e][j] = mfma(vv, pr[n][p], acc[n][e][j]);
            }
        }
        now = next;
        both = both_next;
      }

      // Join the waves: every wave's sums in units of the workgroup's maximum, added through LDS.
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        l[n] = row_sum(l[n]);
        if (g == 0) stat_m[wave][n * 16 + c] = m[n], stat_l[wave][n * 16 + c] = l[n];
      }
      __syncthreads();
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
        for (int x = 1; x < kAttnWaves; ++x) top = fmaxf(top, stat_m[x][n * 16 + c]);
        const float f = exp2_fast(m[n] - top);
        float* mine = join + (wave * 16 + c) * kPitch + g * 16;
#pragma unroll
        for (int e = 0; e < kSets; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (e * 64 + g * 16 + i * 4 >= D) continue;
            f32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = acc[n][e][j][i] * f;
            *reinterpret_cast<f32x4*>(mine + e * 64 + i * 4) = v;
          }
        __syncthreads();
        for (int x = tid; x < 16 * NC; x += kAttnThreads) {
          const int r = x / NC, seg = x - r * NC, row = row0 + n * 16 + r;
          f32x4 o0 = {0, 0, 0, 0}, o1 = {0, 0, 0, 0};
          float rm = stat_m[0][n * 16 + r], rl = 0.0f;
#pragma unroll
          for (int y = 1; y < kAttnWaves; ++y) rm = fmaxf(rm, stat_m[y][n * 16 + r]);
#pragma unroll
          for (int y = 0; y < kAttnWaves; ++y) {
            const float* p = join + (y * 16 + r) * kPitch + seg * 8;
            o0 += *reinterpret_cast<const f32x4*>(p);
            o1 += *reinterpret_cast<const f32x4*>(p + 4);
            rl += stat_l[y][n * 16 + r] * exp2_fast(stat_m[y][n * 16 + r] - rm);
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
        join_parts<D, R, 8, true>(part, args.stats_at, first_wg, parts, min(R, rows - row0), join, finish);
    }
    if (run.left <= 0) return;
    next_job<R>(args, run, me);
    if (run.left <= 0) return;
    __syncthreads();  // the next job's joins use the same LDS
  }
}

}  // namespace ard
