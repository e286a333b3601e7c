// The binary32 form of the attention over packed prompts: 16x16x4 products, whose operands are single values.
//
// Keys in LDS in the order of the operands (1 KB is 16 tokens and 16 of their elements: four products), values as rows,
// read in fours. A round of 32 tokens is on its way while the one before is computed. Bound by the matrix unit:
// a product of 2048 operations takes 32 cycles, and LDS gives an operand for four of them at a time.

#include "ar_prompt.h"

namespace ard {

template <int D_, int NQ_, int WAVES_>
struct PromptF32 {
  static constexpr int DT = DT_F32, D = D_, NQ = NQ_, N = 16, WAVES = WAVES_;
  static constexpr int kSteps = D / 16, kSets = (D + 63) / 64, kTiles = 4 * kSets;
  static constexpr int BYTES = 32 * D * 4;  // of a round's keys, or values
  static constexpr int kAll = BYTES / 1024, kItems = (kAll + WAVES - 1) / WAVES;
  static_assert(offsets_fit(32));
  struct Lds {
    f32x4 keys[2][2][kSteps][64];  // [round's turn][half]
    f32x4 values[2][32][D / 4];
    uint32_t odd[2][WAVES];
  };
  struct Sums {
    f32x4 acc[NQ][kTiles];  // [i] of tile 4 e + j: element 64 e + 16 g + 4 i + j of row c
    float m[NQ], l[NQ];
    // element 64 e + 16 g + y, x = 16 e + y
    __device__ float at(int n, int x) const { return acc[n][(x >> 4) * 4 + (x & 3)][x >> 2 & 3]; }
  };

  Lds& lds;
  uint32_t at;  // of lds
  int wave, lane, c, g;
  uint32_t key_off, value_off[kItems];
  // KB `i` of a wave's: where a round has no multiple of the waves' KB, its last one is moved more than once.
  __device__ int item(int i) const { return min(wave * kItems + i, kAll - 1); }
  __device__ PromptF32(Lds& l, const PromptJob& j, int w, int ln)
      : lds(l), at(static_cast<uint32_t>(reinterpret_cast<uintptr_t>((ARD_LDS Lds*)&l))), wave(w), lane(ln), c(ln & 15), g(ln >> 4) {
    key_off = c * static_cast<uint32_t>(j.k_row) + g * 16;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int x = item(i) * 64 + lane, row = x / (D / 4);
      value_off[i] = row * static_cast<uint32_t>(j.v_row) + (x - row * (D / 4)) * 16;
    }
  }
  __device__ void load(const PromptJob& j, int t, int turn) const {
    const ar::rsrc_t kr = rows_from(j.keys, j.k_row, t, j.end, D * 4), vr = rows_from(j.vals, j.v_row, t, j.end, D * 4);
    const uint32_t to = at + turn * BYTES;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int x = item(i), half = x / kSteps;
      into_lds(to + x * 1024, kr, key_off, half * 16 * static_cast<uint32_t>(j.k_row) + (x - half * kSteps) * 64);
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i)
      into_lds(to + static_cast<uint32_t>(sizeof(lds.keys)) + item(i) * 1024, vr, value_off[i], 0);
  }

  __device__ __forceinline__ void run(const PromptArgs& args, const PromptJob& j, Sums& o) {
    const ar_prompt_attention_args& a = args.a;
    if (j.t_begin < j.t_end) load(j, j.t_begin, 0);
    const PromptRows<NQ> see(j, wave, c);
    f32x4 q[NQ][kSteps];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int i = see.hi[n] - 1;
      const int r = min(wave * (16 * NQ) + n * 16 + c, j.rows - 1 - j.row0);
      const float* x = static_cast<const float*>(a.q) + static_cast<int64_t>(j.q0 + i) * a.q_token +
                       static_cast<int64_t>(j.head * j.group + j.row0 + r - i * j.group) * a.q_head + g * 4;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) q[n][s] = *reinterpret_cast<const f32x4*>(x + s * 16);
      o.m[n] = kLowest, o.l[n] = 0.0f;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) o.acc[n][t] = f32x4{0, 0, 0, 0};
    }

    int turn = 0;
#pragma unroll 1
    for (int t0 = j.t_begin; t0 < j.t_end; t0 += 32, turn ^= 1) {
      ar::wait_vm<0>();
      __syncthreads();  // the round has arrived, and the one before has been read
      if (t0 + 32 < j.t_end) load(j, t0 + 32, turn ^ 1);
      if (t0 + 32 > see.odd_end || t0 < see.odd_begin) {
        const bool some = take_out<DT_F32, 64 * WAVES>(reinterpret_cast<uint8_t*>(lds.values[turn]), BYTES);
        if (lane == 0) lds.odd[turn][wave] = some;
        __syncthreads();
        uint32_t odd = 0;
#pragma unroll
        for (int x = 0; x < WAVES; ++x) odd |= lds.odd[turn][x];
        if (uniform(odd) != 0) {
#pragma unroll 1
          for (int t = t0; t < min(t0 + 32, j.t_end); ++t) {
            int part_of = g;
            asm("" : "+v"(part_of));
#pragma unroll
            for (int e = 0; e < kSets; ++e) {
              if (64 * e + 16 * part_of >= D) continue;
              const f32x4* p = reinterpret_cast<const f32x4*>(j.vals + t * j.v_row) + 16 * e + 4 * part_of;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const f32x4 v = p[i];
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                  for (int n = 0; n < NQ; ++n)
                    if (!(fabsf(v[k]) < INFINITY) && see.sees(n, t)) o.acc[n][4 * e + k][i] += v[k];
              }
            }
          }
        }
      }
      if (t0 >= see.my_end || t0 + 32 <= see.my_begin) continue;
      // Scores.
      f32x4 s[NQ][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n) s[n][0] = s[n][1] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const f32x4 k[2] = {lds.keys[turn][0][i][lane], lds.keys[turn][1][i][lane]};
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int n = 0; n < NQ; ++n) s[n][u] = mfma1(k[u][x], q[n][i][x], s[n][u]);
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n) s[n][0] *= args.scale_log2, s[n][1] *= args.scale_log2;
      if (t0 + 32 > see.whole_end || t0 < see.whole_begin) {
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (!see.sees(n, t0 + (i >> 2) * 16 + g * 4 + (i & 3))) s[n][i >> 2][i & 3] = -INFINITY;
      }
      // Probabilities.
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float top = s[n][0][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = fmaxf(top, s[n][i >> 2][i & 3]);
        if (__any(top > o.m[n] + 8.0f)) {
          const float to = fmaxf(o.m[n], row_max(top));
          const float f = shrink(o.m[n], to);
          o.m[n] = to;
          o.l[n] *= f;
#pragma unroll
          for (int t = 0; t < kTiles; ++t) o.acc[n][t] *= f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = exp2_fast(s[n][i >> 2][i & 3] - o.m[n]);
          o.l[n] += x;
          s[n][i >> 2][i & 3] = x;
        }
      }
      // Values: four elements of token 4 g + x % 4 of half x / 4 at a time.
#pragma unroll
      for (int x = 0; x < 8; ++x)
#pragma unroll
        for (int e = 0; e < kSets; ++e) {
          const f32x4 y = lds.values[turn][(x >> 2) * 16 + g * 4 + (x & 3)][min(e * 16 + c, D / 4 - 1)];
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) o.acc[n][4 * e + k] = mfma1(y[k], s[n][x >> 2][x & 3], o.acc[n][4 * e + k]);
        }
    }
  }
};

template <int D, int NQ, int WAVES, int OCC>
__global__ __launch_bounds__(64 * WAVES, OCC) void prompt_attention_f32(PromptArgs args) {
  prompt_attention<PromptF32<D, NQ, WAVES>>(args);
}

// Bound by the matrix units; waves cover for each other's exponentials and waits, so as many a SIMD as registers and LDS allow.
// With tiles of 64 rows, four workgroups a compute unit end at different times, with tiles of 256 a window's edges and small
// calls cost more. Four prompts of up to 2000 tokens, 16 heads on 2, us:
//   64    4 waves, four times a compute unit   166    (8, twice: 170; 16: 172; 4, twice: 208)
//   96    4, three times       274    (8: 280; 12: 276; 8 of 32 rows: 281)
//   128   8, twice             301    (12: 316; 16: 322; 4, twice: 394)
//   192   12                   462    (8: 480; 4 of 32 rows: 508)
//   256   8                    613    (4: 786)
// A unit takes long here, a job's start and end are soon paid for: us with 1, 3, 6 and 12 units for them, head of 128: 301,
// 313, 341, 359; head of 64, 12 heads on 4, a window of 500: 108, 101, 104, 109.
constexpr int kJobUnits = 2;

PromptKernel select_prompt_f32(int head_dim) {
// rows / 16 of a wave, waves of a workgroup, workgroups of a compute unit
#define ARD_CASE(D, NQ, WAVES, OCC) \
  if (head_dim == D) return {prompt_attention_f32<D, NQ, WAVES, OCC * WAVES / 4>, 256 * OCC, 16 * NQ * WAVES, 64 * WAVES, kJobUnits}
  ARD_CASE(64, 1, 4, 4);
  ARD_CASE(96, 1, 4, 3);
  ARD_CASE(128, 1, 8, 2);
  ARD_CASE(192, 1, 12, 1);
  ARD_CASE(256, 1, 8, 1);
#undef ARD_CASE
  return {nullptr, 0, 0, 0, 0};
}

}  // namespace ard
