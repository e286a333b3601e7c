// Attention over packed prompts (gfx950): causal, grouped heads, each request's keys and values as the
// projection left them.
//
// Mathematics, split of the work and joins as in csrc_decode/ar_decode_attn_rows.h: products transposed, a running maximum, a
// workgroup's waves on 16 * NQ rows each and on the same tokens. Keys and values go from memory into LDS without
// passing through registers; what lies past a request's end arrives as zero by the buffer's bounds and is
// masked like any other. The products are those of ar_prompt_bf16.hip and ar_prompt_f32.hip. Probabilities of bfloat16 calls
// enter the second product as one bfloat16, the row's sum as they are: results are off by up to 0.0021 of their norm, by
// 0.0016 with their own rounding alone (csrc_decode/ar_decode_attn_impl.h has what a second part costs).
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
  int fill, rows, threads;  // workgroups that the device holds, rows of a tile
  int job_units;            // what starting and ending a job costs, in units of 32 tokens
};
PromptKernel select_prompt_bf16(int head_dim, bool large);
PromptKernel select_prompt_f32(int head_dim);
PromptKernel select_prompt_few(int dtype, int head_dim);  // a workgroup a tile and kv head, no workspace

template <int R>
__device__ __forceinline__ Series series_of(const PromptArgs& args, int b) {
  Series c = {0, 0, 0, 0, 1, 0.0, 0, 0};
  const int x = min(b, args.a.nreq - 1);
  const int at = args.a.q_start[x], to = args.a.q_start[x + 1];
  c.q0 = min(max(at, 0), args.a.ntokens);
  c.m = c.kv = b < args.a.nreq ? max(min(to, args.a.ntokens), c.q0) - c.q0 : 0;  // an end may be any number
  c.tiles = static_cast<int>((static_cast<uint32_t>(c.m) * static_cast<uint32_t>(args.group) + R - 1) / R);
  if (c.tiles > 0) {
    auto units = [&](int seen) {
      return ((min(static_cast<uint32_t>(seen), args.most_seen) + args.unit - 1) >> args.unit_shift) + args.job_units;
    };
    c.template set<R>(min(args.tile_tokens, c.m), c.m, args.most_seen, args.group, units);
  }
  return c;
}

// Bytes between two tokens' keys or values, at most: offsets in a round of up to 96 tokens stay below 2^30, and so does
// their sum with those of its end, which the hardware compares with the buffer's size.
constexpr int64_t kMostStride = int64_t(1) << 23;
constexpr bool offsets_fit(int tokens) { return tokens * kMostStride < int64_t(1) << 30; }

// A request's keys or values of one head from token t0 on, as a buffer that ends with its last token; what lies
// beyond reads as zero.
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
typedef short s16x4 __attribute__((ext_vector_type(4)));
// Of 16 lanes that address a row's four elements each, four lanes a row: lane c gets column c of the four rows.
__device__ __forceinline__ u32x2 lds_columns(uint32_t at) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<ARD_LDS s16x4*>(at)));
}

__device__ __forceinline__ f32x4 mfma1(float a, float b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// What a row's sums are worth when its maximum goes from m to `to`. Before the first token they are zeros, but for infinities
// that were added already: times 0 they would become NaN.
__device__ __forceinline__ float shrink(float m, float to) { return m == kLowest ? 1.0f : exp2_fast(m - to); }

// A tile of rows of one request and head, and the tokens that this part of it sees.
struct PromptJob {
  int q0, head, group, rows, row0, i0, rem0, i1;
  float per_group;
  int window, t_begin, t_end, end;
  const uint8_t* keys;  // of the request's first token
  const uint8_t* vals;
  int64_t k_row, v_row;  // bytes between tokens
  // token of row row0 + r: rem0 + r is below 2^17, exact in binary32
  __device__ int token_of(int r) const { return static_cast<int>((rem0 + r + 0.5f) * per_group); }
};

// What a wave's rows see.
template <int NQ>
struct PromptRows {
  int hi[NQ], lo[NQ];
  int my_begin, my_end;        // the tokens that some of them see
  int whole_begin, whole_end;  // those that all see
  int odd_begin, odd_end;      // those that all of the workgroup's see
  __device__ bool sees(int n, int t) const { return t < hi[n] && t >= lo[n]; }
  __device__ PromptRows(const PromptJob& j, int wave, int c) {
    constexpr int RW = 16 * NQ;
    const int last = j.rows - 1 - j.row0;  // rows past the last repeat it
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int i = j.i0 + j.token_of(min(wave * RW + n * 16 + c, last));
      hi[n] = i + 1;
      lo[n] = j.window > 0 ? window_start(i, j.window) : 0;
    }
    const int i_first = j.i0 + j.token_of(min(wave * RW, last)), i_last = j.i0 + j.token_of(min(wave * RW + RW - 1, last));
    my_end = uniform(wave * RW <= last ? min(i_last + 1, j.t_end) : 0);
    my_begin = uniform(j.window > 0 ? max(window_start(i_first, j.window), 0) : 0);
    whole_end = uniform(i_first + 1);
    whole_begin = uniform(j.window > 0 ? window_start(i_last, j.window) : 0);
    odd_end = j.i0 + 1;
    odd_begin = j.window > 0 ? window_start(j.i1, j.window) : 0;
  }
};

// Tiles of 16 * NQ rows a wave; BODY has the products.
template <class BODY>
__device__ __forceinline__ void prompt_attention(const PromptArgs& args) {
  constexpr int D = BODY::D, NQ = BODY::NQ, RW = 16 * NQ, R = RW * BODY::WAVES, DT = BODY::DT, THREADS = 64 * BODY::WAVES;
  constexpr int ES = DT == DT_BF16 ? 2 : 4;
  constexpr int N = BODY::N;  // neighbouring elements of a lane
  __shared__ typename BODY::Lds lds;
  __shared__ int last;

  const ar_prompt_attention_args& a = args.a;
  // consecutive runs on one XCD: workgroups go to the eight in turn
  const int w = (blockIdx.x & 7) * (args.runs >> 3) + (blockIdx.x >> 3);
  Run run;
  Series me;
  int span;
  if (!find_rows<R>(args, w, run, me, span)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const ar::rsrc_t part = ar::make_rsrc(args.part, args.part_bytes);
  PromptJob j;
  j.group = args.group, j.per_group = args.per_group, j.window = a.window;
  j.k_row = a.k_token * ES, j.v_row = a.v_token * ES;
  BODY body(lds, j, wave, lane);

  for (;;) {
    j.q0 = me.q0, j.head = run.head;
    j.rows = me.m * j.group;
    j.row0 = run.tile * R;
    j.i0 = uniform(static_cast<uint32_t>(j.row0) / static_cast<uint32_t>(j.group)), j.rem0 = j.row0 - j.i0 * j.group;
    j.i1 = j.i0 + uniform(j.token_of(min(R, j.rows - j.row0) - 1));
    j.end = j.i1 + 1;
    const int begin = a.window > 0 ? max(window_start(j.i0, a.window), 0) & ~31 : 0;
    const int ntiles = (j.end - begin + 31) >> 5;
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
      j.keys = static_cast<const uint8_t*>(a.k) + me.q0 * j.k_row + run.head * a.k_head * ES;
      j.vals = static_cast<const uint8_t*>(a.v) + me.q0 * j.v_row + run.head * a.v_head * ES;
      j.t_begin = begin + t_first * 32, j.t_end = min(begin + t_last * 32, j.end);
      typename BODY::Sums sums;
      body.run(args, j, sums);

      // This wave's rows are its own: out, or into the workspace. (Places computed anew: kept from job to job they
      // would take the loop's registers.)
      const int here = thread_here() & 63, row = here & 15, own = here >> 4;
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float l = row_sum(sums.l[n]), m = sums.m[n];
        const int r = wave * RW + n * 16 + row;
        if (j.row0 + r < j.rows) {
          const int i = j.i0 + j.token_of(r), head = run.head * j.group + j.row0 + r - i * j.group;
          const int64_t token = me.q0 + i;
          const float f = parts > 1 ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
          const uint32_t at = static_cast<uint32_t>((2 * w + (before == 0)) * R + r);
#pragma unroll
          for (int x = 0; x < BODY::kTiles * 4; x += N) {  // elements 16 (x / N) * N / 4 + N g and on
            const int from = 4 * x + N * own;
            if (from >= D) continue;  // all in the row or none
            float o[N];
#pragma unroll
            for (int y = 0; y < N; ++y) o[y] = sums.at(n, x + y) * f;
            const int64_t to = token * a.o_token + head * a.o_head + from;
#pragma unroll
            for (int y = 0; y < N; y += 4) {
              if (parts > 1)
                ar::st16<ar::kCoh>(part, (at * D + from + y) * 4,
                                   u32x4{__float_as_uint(o[y]), __float_as_uint(o[y + 1]), __float_as_uint(o[y + 2]),
                                         __float_as_uint(o[y + 3])});
              else if constexpr (DT == DT_BF16)
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + to + y) =
                    u32x2{ar::bf16x2_rne(o[y], o[y + 1]), ar::bf16x2_rne(o[y + 2], o[y + 3])};
              else
                *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + to + y) = f32x4{o[y], o[y + 1], o[y + 2], o[y + 3]};
            }
          }
          if (own == 0) {
            if (parts > 1)
              ar::st8<ar::kCoh>(part, args.stats_at + at * 8, u32x2{__float_as_uint(m), __float_as_uint(l)});
            else if (a.lse != nullptr)
              a.lse[token * a.q_heads + head] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;  // l is no denormal
          }
        }
      }
      if (parts > 1) {
        auto finish = [&](int r, int seg, f32x4 o0, f32x4 o1, float top, float rl) {
          const int i = j.i0 + j.token_of(r), head = run.head * j.group + j.row0 + r - i * j.group;
          finish_row<DT>(a, me.q0 + i, head, seg, o0, o1, top, rl);
        };
        if (arrive(args.arrived + first_wg, parts, &last)) {
          const int real = min(R, j.rows - j.row0);
          if (parts == 2) join_few<D, R, 2, 4, true, THREADS>(part, args.stats_at, first_wg, parts, real, finish);
          else if (parts <= 4) join_few<D, R, 4, 2, true, THREADS>(part, args.stats_at, first_wg, parts, real, finish);
          else join_parts<D, R, 8, true, THREADS>(part, args.stats_at, first_wg, parts, real, reinterpret_cast<float*>(&lds), finish);
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
          me = wave_series(series_of<R>(args, run.request));
        } while (me.tiles == 0);
      }
    }
    span = uniform(me.below(run.tile + 1) - me.below(run.tile));
    ar::wait_vm<0>();  // what was on its way into LDS
    __syncthreads();   // the next job uses the same LDS
  }
}

}  // namespace ard
