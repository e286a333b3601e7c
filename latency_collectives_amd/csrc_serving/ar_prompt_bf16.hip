// The bfloat16 form of the attention over packed prompts: 16x16x32 products.
//
// Keys and values go through LDS in rounds of SUB units of 32 tokens, the next round on its way while one is computed. Keys
// lie in the order of the products' operands (1 KB is 16 tokens and 64 bytes of their rows), values as rows, of which the
// transposing reads of LDS make the operands of the second product: a column of four tokens a lane.

#include "ar_prompt.h"

namespace ard {

template <int D_, int NQ_, int WAVES_, int SUB_>
struct PromptBf16 {
  static constexpr int DT = DT_BF16, D = D_, NQ = NQ_, N = 4, WAVES = WAVES_, SUB = SUB_;
  static constexpr int kSteps = D / 32, kTiles = D / 16;
  static constexpr int BYTES = SUB * 32 * D * 2;  // of a round's keys, or values
  static constexpr int kAll = BYTES / 1024, kItems = (kAll + WAVES - 1) / WAVES;
  static constexpr int kPieces = D / 8;  // of 16 bytes, of a row
  static_assert(offsets_fit(SUB * 32));
  struct alignas(256) Lds {
    uint8_t round[2][2][BYTES];
    uint32_t odd[2][WAVES];
  };
  struct Sums {
    f32x4 acc[NQ][kTiles];  // [i] of tile t: element 16 t + 4 g + i of row c
    float m[NQ], l[NQ];
    __device__ float at(int n, int x) const { return acc[n][x >> 2][x & 3]; }
  };

  // Where piece pair `p` (32 bytes, 16 columns) of a row stands: eight rows' 32 bytes fall into different banks
  // (256 bytes) whatever p is. `back`: the other way round.
  __device__ static int place(int p, int row, bool back) {
    constexpr int P = kPieces / 2;
    if (P == 6) {
      const int by = row >> 2 & 1;
      return back ? (p + (by ? 5 : 0)) % 6 : (p + by) % 6;
    }
    return p ^ (P % 8 == 0 ? row & 7 : row >> 1 & 3);  // rows of 128 and 384 bytes: two for the banks' 256
  }

  Lds& lds;
  uint32_t at;  // of lds
  int wave;
  uint32_t key_off, value_off[kItems];  // of a lane, in memory
  uint32_t key_at, value_at;            // in LDS, in the first round
  // (Lanes are counted anew where they are needed outside the loop's straight way.)
  struct Lane {
    int c, g;
    __device__ Lane() { const int t = thread_here(); c = t & 15, g = t >> 4 & 3; }
  };
  // KB `i` of a wave's: where a round has no multiple of the waves' KB, its last one is moved more than once.
  __device__ int item(int i) const { return min(wave * kItems + i, kAll - 1); }
  __device__ PromptBf16(Lds& l, const PromptJob& j, int w, int lane)
      : lds(l), at(static_cast<uint32_t>(reinterpret_cast<uintptr_t>((ARD_LDS Lds*)&l))), wave(w) {
    const int c = lane & 15, g = lane >> 4;
    key_at = at + lane * 16;
    key_off = c * static_cast<uint32_t>(j.k_row) + g * 16;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int x = item(i) * 64 + lane, row = x / kPieces, piece = x - row * kPieces;
      value_off[i] = row * static_cast<uint32_t>(j.v_row) + (place(piece >> 1, row, true) * 2 + (piece & 1)) * 16;
    }
    const int row = g * 4 + (c >> 2);
    value_at = at + BYTES + row * (D * 2) + place(0, row, false) * 32 + (c & 3) * 8;
  }
  // Of tile 0's place, tile t's: the bits that change places are zero in all else of an address.
  __device__ uint32_t tile_at(uint32_t first, int t) const {
    constexpr int P = kPieces / 2, M = P == 6 ? 6 : P % 8 == 0 ? 8 : 4;
    if (P == 6) return first + t * 32 - (t == 5 && (Lane().g & 1) != 0 ? 192 : 0);  // row / 4 is g
    return (first ^ (t % M * 32)) + t / M * (M * 32);
  }
  // Tokens t on and their round's turn; zeros past the end.
  __device__ void load(const PromptJob& j, int t, int turn) const {
    const ar::rsrc_t kr = rows_from(j.keys, j.k_row, t, j.end, D * 2), vr = rows_from(j.vals, j.v_row, t, j.end, D * 2);
    const uint32_t to = at + turn * (2 * BYTES);
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int x = item(k), half = x / kSteps;
      into_lds(to + x * 1024, kr, key_off, half * 16 * static_cast<uint32_t>(j.k_row) + (x - half * kSteps) * 64);
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) into_lds(to + BYTES + item(k) * 1024, vr, value_off[k], 0);
  }

  __device__ __forceinline__ void run(const PromptArgs& args, const PromptJob& j, Sums& o) {
    const ar_prompt_attention_args& a = args.a;
    if (j.t_begin < j.t_end) load(j, j.t_begin, 0);
    const Lane me;
    const PromptRows<NQ> see(j, wave, me.c);
    bf16x8 q[NQ][kSteps];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int i = see.hi[n] - 1;
      const int r = min(wave * (16 * NQ) + n * 16 + me.c, j.rows - 1 - j.row0);
      const uint16_t* x = static_cast<const uint16_t*>(a.q) + static_cast<int64_t>(j.q0 + i) * a.q_token +
                          static_cast<int64_t>(j.head * j.group + j.row0 + r - i * j.group) * a.q_head + me.g * 8;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        q[n][s] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(x + s * 32) ^ args.q_sign);
      o.m[n] = kLowest, o.l[n] = 0.0f;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) o.acc[n][t] = zeros_here();
    }

    int turn = 0;
#pragma unroll 1
    for (int tr = j.t_begin; tr < j.t_end; tr += SUB * 32, turn ^= 1) {
      ar::wait_vm<0>();
      __syncthreads();  // the round has arrived, and the one before has been read
      if (tr + SUB * 32 < j.t_end) load(j, tr + SUB * 32, turn ^ 1);
      if (tr + SUB * 32 > see.odd_end || tr < see.odd_begin) {
        const bool some = take_out<DT_BF16, 64 * WAVES>(lds.round[turn][1], BYTES);
        if ((thread_here() & 63) == 0) lds.odd[turn][wave] = some;
        __syncthreads();
        uint32_t odd = 0;
#pragma unroll
        for (int x = 0; x < WAVES; ++x) odd |= lds.odd[turn][x];
        if (uniform(odd) != 0) {
#pragma unroll 1
          for (int t = tr; t < min(tr + SUB * 32, j.t_end); ++t) {
            const u32x2* p = reinterpret_cast<const u32x2*>(j.vals + t * j.v_row) + Lane().g;
#pragma unroll
            for (int x = 0; x < kTiles; ++x) {
              const u32x2 z = p[4 * x];
              const float v[4] = {bf16_lo(z.x), bf16_hi(z.x), bf16_lo(z.y), bf16_hi(z.y)};
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int n = 0; n < NQ; ++n)
                  if (!(fabsf(v[k]) < INFINITY) && see.sees(n, t)) o.acc[n][x][k] += v[k];
            }
          }
        }
      }
      uint32_t keys_from = key_at + turn * (2 * BYTES);
      asm("" : "+v"(keys_from));  // steps are offsets from it
      const uint32_t values_from = value_at + turn * (2 * BYTES);
      // The first keys of a unit are read before the unit before it ends (128: six, 1535 -> 1500 us; four 1560).
      constexpr int EARLY = 2 * kSteps < 6 ? 2 * kSteps : 6;
      u32x4 kf[EARLY];
      auto read_key = [&](int sub, int i) { return lds_at<u32x4>(keys_from + (sub * 2 * kSteps + (i & 1) * kSteps + (i >> 1)) * 1024); };
      auto read_first = [&](int sub) {
#pragma unroll
        for (int i = 0; i < EARLY; ++i) kf[i] = read_key(sub, i);
      };
      read_first(0);
#pragma unroll
      for (int sub = 0; sub < SUB; ++sub) {
        const int t0 = tr + sub * 32;
        if (t0 >= see.my_end || t0 + 32 <= see.my_begin) {
          if (sub + 1 < SUB) read_first(sub + 1);
          continue;
        }
        // Scores.
        __builtin_amdgcn_s_setprio(1);
        f32x4 s[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) s[n][0] = s[n][1] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const bf16x8 kk = __builtin_bit_cast(bf16x8, k * 2 + u < EARLY ? kf[k * 2 + u] : read_key(sub, k * 2 + u));
#pragma unroll
            for (int n = 0; n < NQ; ++n) s[n][u] = mfma(kk, q[n][k], s[n][u]);
          }
        __builtin_amdgcn_s_setprio(0);
        // The operands of the second product, under way with the probabilities.
        u32x4 vv[kTiles];
        auto read_value = [&](int t) {
          const uint32_t from = tile_at(values_from, t) + sub * (32 * D * 2);
          const u32x2 x = lds_columns(from), y = lds_columns(from + 16 * D * 2);
          vv[t] = u32x4{x.x, x.y, y.x, y.y};
        };
        constexpr int AHEAD = 4;
#pragma unroll
        for (int t = 0; t < AHEAD; ++t) read_value(t);
        __builtin_amdgcn_sched_barrier(0);
        if (t0 + 32 > see.whole_end || t0 < see.whole_begin) {
          const int first = t0 + Lane().g * 4;
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (!see.sees(n, first + (k >> 2) * 16 + (k & 3))) s[n][k >> 2][k & 3] = -INFINITY;
        }
        // Probabilities.
        bf16x8 pr[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          float top = s[n][0][0];
#pragma unroll
          for (int k = 1; k < 8; ++k) top = fmaxf(top, s[n][k >> 2][k & 3]);
          top *= args.scale_log2;
          if (__any(top > o.m[n] + 8.0f)) {
            const float to = fmaxf(o.m[n], row_max(top));
            const float f = shrink(o.m[n], to);
            o.m[n] = to;
            o.l[n] *= f;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) o.acc[n][t] *= f;
          }
          float x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            x[k] = exp2_fast(fmaf(s[n][k >> 2][k & 3], args.scale_log2, -o.m[n]));
            o.l[n] += x[k];
          }
          split<1>(x, &pr[n]);
        }
        // Values.
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if (t >= AHEAD) read_value(t);
          if (t == kTiles / 2 && sub + 1 < SUB) read_first(sub + 1);
#pragma unroll
          for (int n = 0; n < NQ; ++n) o.acc[n][t] = mfma(__builtin_bit_cast(bf16x8, vv[t]), pr[n], o.acc[n][t]);
        }
      }
    }
  }
};

template <int D, int NQ, int WAVES, int SUB, int OCC>
__global__ __launch_bounds__(64 * WAVES, OCC) void prompt_attention_bf16(PromptArgs args) {
  prompt_attention<PromptBf16<D, NQ, WAVES, SUB>>(args);
}

// What bounds it: a unit of 32 tokens and 32 rows of 128 takes the matrix units 512 cycles and the others about 600 (one
// exponential a score, a comparison, conversions), so waves have to cover for each other: three a SIMD, as many as their
// registers allow with 32 rows each. Four prompts of up to 8000 tokens, 16 query heads on 4, TFLOP/s:
//   64    8 waves of 32 rows, twice a compute unit   845    (12, once: 787)
//   96    12 of 32     970    (8: 767)
//   128   12 of 32     1057   (8 of 32: 845; six prompts of up to 8191, 32 heads on 8, 1050, and 8 of 16 twice 820)
//   192   8 of 32      985    (12 of 16: 910)
//   256   12 of 16     873    (8 of 16: 720)
// A head of 64 has half the products of one of 128 for the same exponentials; rows of 192 and 256 leave a wave registers for fewer
// rows (256: 16, so that an operand from LDS feeds one product) or a SIMD for fewer waves (192: two).
// Smaller calls, where a workgroup's own rows and the joins count for more: 8 waves of 16 rows, twice a compute unit.
// Six prompts of up to 8191 tokens, 32 heads on 8, us with a job's start and end taken for 2, 4, 6, 8 and 12 units: 1679, 1612,
// 1560, 1551, 1567 (head of 256, four of up to 8000: 1446, 1371, 1318, 1291, 1302).
constexpr int kJobUnits = 8;

PromptKernel select_prompt_bf16(int head_dim, bool large) {
// rows / 16 of a wave, waves of a workgroup, units of a round, workgroups of a compute unit
#define ARD_CASE(D, NQ, WAVES, SUB, OCC) \
  if (head_dim == D) return {prompt_attention_bf16<D, NQ, WAVES, SUB, OCC * WAVES / 4>, 256 * OCC, 16 * NQ * WAVES, 64 * WAVES, kJobUnits}
  if (large) {
    ARD_CASE(64, 2, 8, 2, 2);
    ARD_CASE(96, 2, 12, 3, 1);
    ARD_CASE(128, 2, 12, 3, 1);
    ARD_CASE(192, 2, 8, 2, 1);
  } else {
    ARD_CASE(64, 1, 8, 2, 2);
    ARD_CASE(96, 1, 8, 2, 2);
    ARD_CASE(128, 1, 8, 2, 2);
    ARD_CASE(192, 1, 8, 1, 2);
  }
  ARD_CASE(256, 1, 12, 2, 1);
#undef ARD_CASE
  return {nullptr, 0, 0, 0, 0};
}

}  // namespace ard
