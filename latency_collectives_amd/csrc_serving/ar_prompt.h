// Attention over packed prompts (gfx950): causal, grouped heads, each request's keys and values as the
// projection left them.
//
// Mathematics, split of the work and joins as in csrc_decode/ar_decode_attn_rows.h: products transposed, a running maximum, a
// workgroup's four waves on 16 * NQ rows each and on the same tokens. Keys and values go from memory into LDS without
// passing through registers, a round (SUB units of 32 tokens) ahead; what lies past a request's end
// arrives as zero by the buffer's bounds and is masked like any other.
//
//   keys       in the order of the product's operands: 1 KB is 16 tokens and 64 bytes of their rows
//   values     as rows. bfloat16: the operand of the second product is a column of eight tokens, two of the
//              transposing reads of LDS; pairs of 16-byte pieces change places within a row so that the 16
//              rows of a read fall into different banks. binary32 (16x16x4 products, whose operands
//              are single values): in fours along a row.
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

// 64 lanes' 16 bytes each, at voffset + soffset of the buffer, into LDS at `to` and on, in the lanes' order. The
// compiler does not count them: wait_vm before the barrier that hands them over. (An SGPR that a vector
// instruction wrote has to be five wait states old, M0 one.)
__device__ __forceinline__ void into_lds(uint32_t to, ar::rsrc_t from, uint32_t voffset, uint32_t soffset) {
  asm volatile("s_nop 4\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(to), "v"(voffset), "s"(from), "s"(soffset)
               : "memory", "m0");
}
#define ARD_LDS __attribute__((address_space(3)))
template <class T>
__device__ __forceinline__ T lds_at(uint32_t at) {
  return *reinterpret_cast<const ARD_LDS T*>(at);
}
typedef short s16x4 __attribute__((ext_vector_type(4)));
// Of 16 lanes that address a row's four elements each, four lanes a row: lane c gets column c of the four rows.
__device__ __forceinline__ u32x2 lds_columns(uint32_t at) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<ARD_LDS s16x4*>(at)));
}

// A round of tokens in LDS: keys, then values, BYTES each.
template <int DT, int D, int SUB>
struct Round {
  static constexpr bool kBf16 = DT == DT_BF16;
  static constexpr int ES = kBf16 ? 2 : 4;
  static constexpr int BYTES = SUB * 32 * D * ES;
  static constexpr int kSteps = D * ES / 64;                 // KB of 16 tokens' keys
  static constexpr int kItems = BYTES / 1024 / kAttnWaves;   // KB that a wave moves, of either
  static constexpr int kPieces = D * ES / 16;                // of a row
  static_assert(BYTES % (1024 * kAttnWaves) == 0 && kItems * kAttnWaves == SUB * 2 * kSteps);

  // Where piece pair `p` (32 bytes, 16 columns) of a bfloat16 row stands: eight rows' 32 bytes fall into
  // different banks (256 bytes) whatever p is. `back`: the other way round.
  __device__ static int place(int p, int row, bool back) {
    if (!kBf16) return p;
    constexpr int P = kPieces / 2;
    if (P == 6) {
      const int by = row >> 2 & 1;
      return back ? (p + (by ? 5 : 0)) % 6 : (p + by) % 6;
    }
    return p ^ (P % 8 == 0 ? row & 7 : row >> 1 & 3);  // rows of 128 and 384 bytes: two of a bank's turn
  }

  uint32_t key_off, value_off[kItems];  // of a lane, in the round's buffers
  __device__ void setup(uint32_t k_row, uint32_t v_row, int wave, int lane) {
    const int c = lane & 15, g = lane >> 4;
    key_off = (first_half(wave) * 16 + c) * k_row + g * 16;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int at = (wave * kItems + i) * 64 + lane, row = at / kPieces, piece = at - row * kPieces;
      value_off[i] = row * v_row + (place(piece >> 1, row, true) * 2 + (piece & 1)) * 16;
    }
  }
  // A wave's keys: whole halves where there are four or more, else half of one's steps.
  static constexpr int kHalves = SUB * 2 >= kAttnWaves ? SUB * 2 / kAttnWaves : 1;
  static constexpr int kMySteps = kItems / kHalves;
  __device__ static int first_half(int wave) { return SUB * 2 >= kAttnWaves ? wave * kHalves : wave % (SUB * 2); }
  __device__ static int first_step(int wave) { return SUB * 2 >= kAttnWaves ? 0 : wave / (SUB * 2) * kMySteps; }
  __device__ void load(uint32_t lds, ar::rsrc_t kr, ar::rsrc_t vr, uint32_t k_row, int wave) const {
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int s = 0; s < kMySteps; ++s)
        into_lds(lds + ((first_half(wave) + h) * kSteps + first_step(wave) + s) * 1024, kr, key_off,
                 h * 16 * k_row + (first_step(wave) + s) * 64);
#pragma unroll
    for (int i = 0; i < kItems; ++i) into_lds(lds + BYTES + (wave * kItems + i) * 1024, vr, value_off[i], 0);
  }
};

__device__ __forceinline__ f32x4 mfma1(float a, float b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

template <int DT, int D, int NQ, int SUB, int OCC>
__global__ __launch_bounds__(kAttnThreads, OCC) void prompt_attention(PromptArgs args) {
  constexpr int RW = 16 * NQ, R = RW * kAttnWaves;
  constexpr bool kBf16 = DT == DT_BF16;
  constexpr int ES = kBf16 ? 2 : 4;
  typedef Round<DT, D, SUB> Stage;
  constexpr int kSteps = Stage::kSteps, kSets = (D + 63) / 64;
  // bfloat16: tile t has elements 16 t + 4 g + i of row c in [i]; binary32: 64 (t / 4) + 16 g + 4 i + t % 4.
  constexpr int kTiles = kBf16 ? D / 16 : 4 * kSets;
  typedef typename std::conditional<kBf16, bf16x8, f32x4>::type Q;  // a lane's elements of a step
  constexpr bool kAhead = kBf16 && D <= 192;  // the next unit's keys are read behind this one's scores
  constexpr int kValuesAhead = kBf16 ? (D <= 128 ? D / 16 : 4) : 0;  // values read behind them
  __shared__ __attribute__((aligned(1024))) uint8_t tokens[2][2 * Stage::BYTES];
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
  const uint32_t lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((ARD_LDS uint8_t*)&tokens[0][0]));
  Stage stage;
  stage.setup(static_cast<uint32_t>(k_row), static_cast<uint32_t>(v_row), wave, lane);
  // A lane's places in a round's LDS.
  uint32_t key_at = lds + lane * 16;
  uint32_t value_at[kBf16 ? kTiles : 1];
#pragma unroll
  for (int t = 0; t < (kBf16 ? kTiles : 1); ++t) {
    const int row = g * 4 + (kBf16 ? c >> 2 : 0);
    value_at[t] = lds + Stage::BYTES + row * (D * ES) + (kBf16 ? Stage::place(t, row, false) * 32 + (c & 3) * 8 : 0);
  }
  int turn = 2 * Stage::BYTES;  // from one round's LDS to the other's
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
      auto load = [&](uint32_t to, int t) {
        stage.load(to, rows_from(keys, k_row, t, end, D * ES), rows_from(vals, v_row, t, end, D * ES),
                   static_cast<uint32_t>(k_row), wave);
      };
      // LDS of the round that is read next (key_at's), and its turn among any_odd's.
      const auto now_at = [&] { return uniform(static_cast<int>(key_at - lane * 16)); };
      const auto now = [&] { return turn < 0; };
      // Rounds that some row sees in part: from the first row's end on, and up to the last one's window.
      const int odd_begin = a.window > 0 ? window_start(i1, a.window) : 0;
      if (t_begin < t_end) load(now_at(), t_begin);

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

      f32x4 acc[NQ][kTiles];
      float m[NQ], l[NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        m[n] = kLowest, l[n] = 0.0f;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) acc[n][t] = f32x4{0, 0, 0, 0};
      }

      for (int tr = t_begin; tr < t_end; tr += SUB * 32) {
        ar::wait_vm<0>();
        __syncthreads();  // the round has arrived, and the one before has been read
        const bool more = tr + SUB * 32 < t_end;
        auto keys_of = [&](int sub, int x) { return __builtin_bit_cast(Q, lds_at<u32x4>(key_at + (sub * 2 * kSteps + x) * 1024)); };
        Q kk[kAhead ? 2 * kSteps : 1];
        if (kAhead)
#pragma unroll
          for (int x = 0; x < 2 * kSteps; ++x) kk[x] = keys_of(0, x);
        if (more) load(now_at() + turn, tr + SUB * 32);
        if (tr + SUB * 32 > i0 + 1 || tr < odd_begin) {
          // Infinities and NaN that not all rows see: taken out of the round, and added for the rows that do.
          uint32_t* const mine = reinterpret_cast<uint32_t*>(tokens[now()] + Stage::BYTES) + tid * 4;
          bool some = false;
          for (int x = 0; x < Stage::BYTES / 16; x += kAttnThreads) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(mine + x * 4);
            u32x4 y = v;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if constexpr (kBf16) y[i] = finite_only(v[i]);
              else y[i] = (v[i] & 0x7F800000u) == 0x7F800000u ? 0 : v[i];
            }
            if (y[0] != v[0] || y[1] != v[1] || y[2] != v[2] || y[3] != v[3]) {
              some = true;
              *reinterpret_cast<u32x4*>(mine + x * 4) = y;
            }
          }
          some = __any(some);
          if (lane == 0) reinterpret_cast<uint32_t*>(&any_odd[now()])[wave] = some;
          __syncthreads();
          const u32x4 odd = any_odd[now()];
          if (uniform(odd[0] | odd[1] | odd[2] | odd[3]) != 0) {
            const int upto = min(tr + SUB * 32, t_end);
#pragma unroll 1
            for (int t = tr; t < upto; ++t) {
              const uint8_t* row = vals + t * v_row;
              int part_of = g;
              asm("" : "+v"(part_of));
#pragma unroll
              for (int x = 0; x < kTiles; ++x) {
                if (!kBf16 && (x & 3) != 0) continue;
                float v[16];
                constexpr int N = kBf16 ? 4 : 16;
                const int from = 16 * x + N * part_of;
                if (from >= D) continue;
#pragma unroll
                for (int i = 0; i < N; i += 4) {
                  if constexpr (kBf16) {
                    const u32x2 z = *reinterpret_cast<const u32x2*>(row + from * 2);
                    v[0] = bf16_lo(z.x), v[1] = bf16_hi(z.x), v[2] = bf16_lo(z.y), v[3] = bf16_hi(z.y);
                  } else {
                    const f32x4 z = *reinterpret_cast<const f32x4*>(row + (from + i) * 4);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i + j] = z[j];
                  }
                }
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                  for (int i = 0; i < N; ++i)
                    if (!(fabsf(v[i]) < INFINITY) && t < hi[n] && t >= lo[n])
                      acc[n][kBf16 ? x : x + (i & 3)][kBf16 ? i : i >> 2] += v[i];
              }
            }
          }
        }
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub) {
          const int t0 = tr + sub * 32;
          const bool mine = t0 < my_end && t0 + 32 > my_begin;
          f32x4 s[NQ][2];
          u32x4 vv[kBf16 ? kTiles : 1];
          auto values_of = [&](int t) {
            const uint32_t at = value_at[kBf16 ? t : 0] + sub * (32 * D * ES);
            const u32x2 x = lds_columns(at), y = lds_columns(at + 16 * D * ES);
            return u32x4{x.x, x.y, y.x, y.y};
          };
          if (mine) {
            // Scores.
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int n = 0; n < NQ; ++n) s[n][0] = s[n][1] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int i = 0; i < kSteps; ++i) {
                const Q k1 = kAhead ? kk[u * kSteps + i] : keys_of(sub, u * kSteps + i);
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                  if constexpr (kBf16) {
                    s[n][u] = mfma(k1, q[n][i], s[n][u]);
                  } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[n][u] = mfma1(k1[j], q[n][i][j], s[n][u]);
                  }
                }
              }
            __builtin_amdgcn_s_setprio(0);
            // The operands of the second product, under way with the probabilities.
            if constexpr (kBf16) {
#pragma unroll
              for (int t = 0; t < kValuesAhead; ++t) vv[t] = values_of(t);
            }
          }
          if (kAhead && sub + 1 < SUB)
#pragma unroll
            for (int x = 0; x < 2 * kSteps; ++x) kk[x] = keys_of(sub + 1, x);
          if (!mine) continue;
          __builtin_amdgcn_sched_barrier(0);
          if (!kBf16)
#pragma unroll
            for (int n = 0; n < NQ; ++n) s[n][0] *= args.scale_log2, s[n][1] *= args.scale_log2;
          if (t0 + 32 > whole_end || t0 < whole_begin) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int t = t0 + u * 16 + g * 4 + i;
                  if (t >= hi[n] || t < lo[n]) s[n][u][i] = -INFINITY;
                }
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
              for (int t = 0; t < kTiles; ++t) acc[n][t] *= f;
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
            for (int t = 0; t < kTiles; ++t) {
              if (t >= kValuesAhead) vv[t] = values_of(t);
#pragma unroll
              for (int n = 0; n < NQ; ++n) acc[n][t] = mfma(__builtin_bit_cast(bf16x8, vv[t]), pr[n], acc[n][t]);
            }
          } else {
#pragma unroll
            for (int x = 0; x < 8; ++x)
#pragma unroll
              for (int e = 0; e < kSets; ++e) {
                // four elements of token 4 g + x % 4 of half x / 4
                const f32x4 y = lds_at<f32x4>(value_at[0] + (sub * 32 + (x >> 2) * 16 + (x & 3)) * (D * 4) + min(e * 64 + c * 4, D - 4) * 4);
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                  for (int j = 0; j < 4; ++j) acc[n][4 * e + j] = mfma1(y[j], s[n][x >> 2][x & 3], acc[n][4 * e + j]);
              }
          }
        }
        key_at += turn;
#pragma unroll
        for (int t = 0; t < (kBf16 ? kTiles : 1); ++t) value_at[t] += turn;
        turn = -turn;
      }

      // This wave's rows are its own: out, or into the workspace. (Places computed anew: kept from job to job they
      // would take the loop's registers.)
      int own = g;
      asm("" : "+v"(own));
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        l[n] = row_sum(l[n]);
        const int r = wave * RW + n * 16 + c;
        if (row0 + r < rows) {
          const int i = i0 + token_of(r), head = run.head * group + row0 + r - i * group;
          const int64_t token = me.q0 + i;
          const float f = parts > 1 ? 1.0f : l[n] == 0.0f ? 0.0f : 1.0f / l[n];
          const uint32_t at = static_cast<uint32_t>((2 * w + (before == 0)) * R + r);
          constexpr int N = kBf16 ? 4 : 16;  // neighbouring elements of a lane
#pragma unroll
          for (int x = 0; x < kTiles; x += kBf16 ? 1 : 4) {
            const int from = 16 * x + N * own;
            if (from >= D) continue;  // all in the row or none
            float o[N];
#pragma unroll
            for (int y = 0; y < N; ++y) o[y] = (kBf16 ? acc[n][x][y & 3] : acc[n][x + (y & 3)][y >> 2]) * f;
            const int64_t to = token * a.o_token + head * a.o_head + from;
#pragma unroll
            for (int y = 0; y < N; y += 4) {
              if (parts > 1)
                ar::st16<ar::kCoh>(part, (at * D + from + y) * 4,
                                   u32x4{__float_as_uint(o[y]), __float_as_uint(o[y + 1]), __float_as_uint(o[y + 2]),
                                         __float_as_uint(o[y + 3])});
              else if constexpr (kBf16)
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + to) = u32x2{ar::bf16x2_rne(o[0], o[1]), ar::bf16x2_rne(o[2], o[3])};
              else
                *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + to + y) = f32x4{o[y], o[y + 1], o[y + 2], o[y + 3]};
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
