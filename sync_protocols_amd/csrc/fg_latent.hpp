// Latent attention, absorbed form, of one new token over a paged cache of rows
// [latent of R | rope of P], one for all heads:
//   a[b][h] = W_k[h]^T q_nope[b][h]                         absorb_kernel
//   u[b][h] = sum_t w_t c_t,  w = softmax of scale (a . c_t + q_rope . r_t)       latent_kernel
//   out[b][h] = W_v[h] u[b][h]                              values_product_kernel
// Keys and values are the same rows, so a row is read once, for up to 128 heads:
// 2 H (2 R + P) flops for 2 (R + P) bytes, 242 a byte with 128 heads of 512 + 64, near the ratio of the matrix to the memory rate.
//
// latent_kernel: tiles of T rows go to LDS by direct loads, two tiles in turn,
// and serve both products as 16x16x32 matrix instructions with the head in the lane:
//   S^T[token][head] = C A^T       C: 16 bytes of a row
//   U^T[dim][head] += C^T W^T      C^T by transposing reads: 4 tokens of a dim in a lane,
//                                  the tokens of the lane's own scores
// LDS gives at most 128 bytes a clock, so what is read from it has to serve many heads
// (16 heads a wave, all rows and columns each: 64 requests, 128 heads 122 us; as follows 116, and 105 with the steps noted below): two waves share
// 16 HW heads, each takes half of the rows for the scores and half of the columns for the sum. Their weights change places through
// LDS, 16 bytes a lane, as operands of the second product; each wave holds all of A's columns in registers.
// Chunks of 16 bytes lie permuted in a row, so that what a read takes from 16 (8) rows falls on different banks.
#pragma once

#include "fg_paged.hpp"

namespace fg {
namespace ops {

struct LatentArgs {
  SplitArgs split;
  const char* a;                     // absorbed queries with their rope part: bf16 [batch][heads][R + P]
  const char* cache;
  uint16_t* mean;                    // [batch][heads][2][R], see put_mean
  float* lse;
  float* part;                       // [places][head tiles][R / 16][64 lanes][4]: sums as the instructions leave them
  float* ml;                         // [places][16 head tiles][2]
  int64_t rest;                      // bytes from the queries to their rests (kQueryPairs)
  int64_t c_page, lse_b;             // bytes, elements
  int32_t c_tok, heads, tiles, parts;           // 16-head tiles; parts: workgroups that share rows, each with other heads
  float c;
};

constexpr int kKeysAhead = 3, kValuesAhead = 4;  // reads of LDS in flight before the products that take them

// Direct loads to LDS are in flight across barriers: those wait for what LDS itself has to finish, and for the loads only where asked.
// (__syncthreads() waits for both.)
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void loads_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The weighted mean as two bf16 numbers, [batch][heads][2][R]: one would add an error as large as the result's own rounding.
__device__ __forceinline__ void put_mean(uint16_t* to, int R, f32x4 y) {
  *(u32x2*)to = u32x2{f2_bf16(y[0], y[1]), f2_bf16(y[2], y[3])};
  *(u32x2*)(to + R) = u32x2{f2_bf16(bf16_rest(y[0]), bf16_rest(y[1])), f2_bf16(bf16_rest(y[2]), bf16_rest(y[3]))};
}

// G groups of 16 HW heads, two waves each.
template <int R, int P, int G, int HW>
struct LatentShape {
  static constexpr int W = 2 * G;               // waves
  static constexpr int NB = W, T = 16 * NB;     // blocks of 16 rows of a tile: a wave loads one
  static constexpr int B = NB / 2;              // blocks whose scores a wave forms
  static constexpr int NC = (R + P) / 8;        // chunks of a row
  static constexpr int KS = (R + P) / 32;       // matrix instructions of a score
  static constexpr int LOADS = NC / 4;          // of 64 chunks for 16 rows
  static constexpr int ROW = 2 * (R + P);
  static constexpr int TILE = T * ROW;
  static constexpr int WEIGHTS = 2 * TILE;      // in LDS: [G][HW][N2][NB][64 lanes] packed weights of 4 rows, ...
  // A weight as two bf16 numbers where the matrix instructions wait for memory anyway: 131072 tokens with 16 heads take the same 33.5 us, and 1001
  // tokens come out 0.0025 off instead of 0.0028 (0.0017 is the result's own rounding). With four waves LDS has no room for them.
  static constexpr int N2 = G == 1 ? 2 : 1;
  // The same for the absorbed queries where registers have room for it, one tile of 16 heads: nothing but the result's own rounding is left
  // (35 us; 1001 tokens 7.1 instead of 6.8).
  static constexpr bool kQueryPairs = G * HW == 1;
  static constexpr int HIGHS = WEIGHTS + N2 * G * HW * NB * 512;  // ... largest scores [G][2][HW][16], ...
  static constexpr int FLAGS = HIGHS + G * HW * 128;         // ... and whether a wave found one that raises the maximum
  static constexpr int LDS = FLAGS + 4 * W;
  static_assert(NC % 16 == 8 || NC % 16 == 4, "row");
  static constexpr int COLS = R / 2, J = COLS / 16;          // a wave's columns of the sum
  // Place of chunk c in row t. A row is 8 (or 4) chunks past a multiple of 16, 256 bytes, so rows of one parity (of one t % 4) share a half
  // (a quarter) of the banks; in it the 16 rows of a key read, and the 8 rows of which a transposing read takes 32 bytes, get different ones.
  static constexpr bool kHalves = NC % 16 == 8;
  static __device__ __forceinline__ uint32_t place(uint32_t c, uint32_t t) {
    return c ^ (kHalves ? (t & 6) | (t >> 3 & 1) : (t >> 1 & 2) | (t >> 3 & 1));
  }
  // The same for what the products read, as a few addresses per lane plus constants: chunk 4 ks + quarter of rows 16 i + m, ...
  static constexpr int kKeyBases = kHalves ? 2 : 1, kValueBases = kHalves ? 4 : 2;
  static __device__ __forceinline__ int key_base(int e, int m, int quarter) { return m * ROW + 16 * place(4 * e + quarter, m); }
  static constexpr int key_offset(int i, int ks) { return 16 * i * ROW + 64 * (ks / kKeyBases * kKeyBases); }
  // ... and columns 16 j + 4 (m % 4) + 0..3 of the wave's share of row 16 i + 4 quarter + m / 4, of which a transposing read makes
  // rows 4 quarter + 0..3 of column 16 j + m
  static __device__ __forceinline__ int value_base(int e, int m, int quarter, int part) {
    const int row = 4 * quarter + (m >> 2);
    return row * ROW + 2 * COLS * part + 16 * place(2 * e + (m >> 1 & 1), row) + 8 * (m & 1);
  }
  static constexpr int value_offset(int i, int j) { return 16 * i * ROW + 32 * (j / kValueBases * kValueBases); }
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
__device__ __forceinline__ u32x2 read_turned(const char* from) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)from));
}

// 16 bytes a lane from base + off to LDS at `to`, 64 lanes side by side. In assembly, because the compiler lets transposing reads wait for every
// direct load that it knows of; these have no result registers, and loads_barrier() waits for them.
// m0 is named so that nothing of the compiler's own is kept in it; it warns of any reserved register there.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t off, const char* to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(__builtin_amdgcn_readfirstlane((int)(uintptr_t)(__attribute__((address_space(3))) const char*)to)),
               "v"(off), "s"(base)
               : "m0");
}
#pragma clang diagnostic pop

// The rows of a workgroup's pieces, tile after tile, for the direct loads, which run one tile ahead of the products. Page and
// place of 64 blocks are in the lanes; those of the next ones, or of the next piece, are asked for with the tile before.
template <class Sh>
struct RowTiles {
  static constexpr int T = Sh::T, NB = Sh::NB, LIST = 64 / NB;
  static constexpr uint32_t kFull = NB == 4 ? 0x10101010u : 0x1010u;
  Pieces<T> p;
  const char* from;                  // of this wave's block
  int32_t page, at;
  int t, tiles;                      // of the piece
  bool more;
  __device__ __forceinline__ void fetch(const SplitArgs& s, int lane) {
    const uint32_t tok = (uint32_t)p.begin + T * (uint32_t)t + 16 * (uint32_t)lane, i = tok / (uint32_t)s.page;
    at = (int32_t)(tok - i * (uint32_t)s.page);
    page = tok < (uint32_t)p.len ? s.table[p.b * s.ldt + i] : -1;          // not behind the last token
  }
  __device__ __forceinline__ void enter(const SplitArgs& s, int lane) {       // the piece p, or the first one after it that has rows
    more = true;
    t = 0;
    while ((tiles = steps_of<T>(p.end - p.begin)) == 0)
      if (!p.next(s, 1)) {
        more = false;
        return;
      }
    fetch(s, lane);
  }
  // The next tile: where this wave's block lies, and the rows of each block, 8 bits each. Behind the last tile: some rows of the cache.
  __device__ __forceinline__ uint32_t find_rows(const LatentArgs& a, int wave) {
    const int left = p.len - p.begin - T * t, l = NB * (t & (LIST - 1));
    uint32_t seen = 0;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const uint32_t id = __builtin_amdgcn_readlane(page, l + i);
      seen |= (uint32_t)(id < (uint32_t)a.split.n_pages ? max(0, min(left - 16 * i, 16)) : 0) << (8 * i);
    }
    const bool there = more && (seen >> (8 * wave) & 255) != 0;
    const int64_t id = there ? __builtin_amdgcn_readlane(page, l + wave) : 0, row = there ? __builtin_amdgcn_readlane(at, l + wave) : 0;
    from = a.cache + id * a.c_page + row * a.c_tok;
    ++t;
    return seen;
  }
  // The i-th of its Sh::LOADS loads. A wave that asks for more than the unit takes waits until it may, so they are asked for one by one between
  // the products (340 clocks of a tile's 7600 are left to wait for them).
  uint32_t off[Sh::LOADS];
  __device__ __forceinline__ void set(const LatentArgs& a, int lane) {
#pragma unroll
    for (int i = 0; i < Sh::LOADS; ++i) {
      const uint32_t slot = 64 * i + lane, row = slot / Sh::NC;
      off[i] = row * (uint32_t)a.c_tok + 16 * Sh::place(slot - row * Sh::NC, row);
    }
  }
  __device__ __forceinline__ void load(char* to, int i, int wave) const { load_to_lds(from, off[i], to + 1024 * (Sh::LOADS * wave + i)); }
  // After the loads: on to the tile after it.
  __device__ __forceinline__ void step(const SplitArgs& s, int lane) {
    if (t == tiles) {
      if (p.next(s, 1)) enter(s, lane);
      else more = false;
    } else if ((t & (LIST - 1)) == 0) {
      fetch(s, lane);
    }
  }
};

template <int R, int P, int G, int HW>
__global__ __launch_bounds__(128 * G) void latent_kernel(LatentArgs a) {
  typedef LatentShape<R, P, G, HW> Sh;
  constexpr int W = Sh::W, T = Sh::T, NB = Sh::NB, B = Sh::B, KS = Sh::KS, NC = Sh::NC, J = Sh::J, N2 = Sh::N2;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ SplitShared sh;
  // workgroups go round the 8 dies: those of one share of the work are on one die, and its rows in that die's L2
  const int turn = blockIdx.x >> 3, head_part = turn % a.parts;
  const int lane = threadIdx.x & 63, m = lane & 15, quarter = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowTiles<Sh> rows;
  if (!rows.p.template find<64 * W>(a.split, turn / a.parts * 8 + (blockIdx.x & 7), sh)) return;
  Pieces<T> p = rows.p;
  const int group = wave >> 1, part = wave & 1;
  const int tile16 = HW * (G * head_part + group);             // the first of this wave's tiles of 16 heads
  u32x2* const weights = (u32x2*)(lds + Sh::WEIGHTS) + group * (N2 * HW * NB * 64) + lane;
  float* const highs = (float*)(lds + Sh::HIGHS) + group * (2 * HW * 16) + m;
  int32_t* const flags = (int32_t*)(lds + Sh::FLAGS);
  int key_at[Sh::kKeyBases], value_at[Sh::kValueBases];
#pragma unroll
  for (int e = 0; e < Sh::kKeyBases; ++e) key_at[e] = Sh::key_base(e, m, quarter);
#pragma unroll
  for (int e = 0; e < Sh::kValueBases; ++e) value_at[e] = Sh::value_base(e, m, quarter, part);

  int g = 0;                           // tiles so far
  uint32_t seen = 0, coming = 0;       // rows of the tile at hand, and of the one that is loaded beside it
  rows.set(a, lane);
  rows.enter(a.split, lane);
  if (rows.more) {
    seen = rows.find_rows(a, wave);
#pragma unroll
    for (int i = 0; i < Sh::LOADS; ++i) rows.load(lds, i, wave);
    rows.step(a.split, lane);
    coming = rows.find_rows(a, wave);
  }
  // The queries of all heads of the workgroup, through the buffer that no rows are coming to. One load after the other: unrolled, their addresses
  // spilled what the tiles need (64 requests, 128 heads: 117 us instead of 105).
  auto ask_queries = [&] {
    if (wave >= (Sh::kQueryPairs ? 2 : G * HW)) return;
    const int first = 16 * (HW * G * head_part + (Sh::kQueryPairs ? 0 : wave));
    const char* from = a.a + (Sh::kQueryPairs && wave == 1 ? a.rest : 0) + ((int64_t)p.b * a.heads + min(first, a.heads - 1)) * Sh::ROW;
#pragma unroll 1
    for (int i = 0; i < Sh::LOADS; ++i) {
      const int slot = 64 * i + lane, row = slot / NC, there = max(0, min(row, a.heads - 1 - first));
      load_to_lds(from, there * Sh::ROW + 16 * Sh::place(slot - row * NC, row), lds + (~g & 1) * Sh::TILE + 1024 * (Sh::LOADS * wave + i));
    }
  };
  ask_queries();
  bool stored = false;                 // stores of the last piece's sums were asked for after the queries
  for (;;) {
    bf16x8 q[HW][KS], rest[Sh::kQueryPairs ? R / 32 : 1];
    f32x4 o[HW][J];
    float top[HW], l[HW];
    {
      char* const buffer = lds + (~g & 1) * Sh::TILE;
      // The queries are there, and the rows that were asked for before them; the stores may be under way (waiting for them too: 123 us for 117).
      if (stored) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(HW * J) : "memory");
      else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      lds_barrier();
#pragma unroll
      for (int ht = 0; ht < HW; ++ht) {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          u32x4 w = *(const u32x4*)(buffer + key_at[s % Sh::kKeyBases] + Sh::key_offset(0, s) + 16 * Sh::ROW * (HW * group + ht));
          if (16 * (tile16 + ht) + m >= a.heads) w = u32x4{0u, 0u, 0u, 0u};
          q[ht][s] = __builtin_bit_cast(bf16x8, w);
          if constexpr (Sh::kQueryPairs) {
            if (s >= R / 32) continue;
            w = *(const u32x4*)(buffer + key_at[s % Sh::kKeyBases] + Sh::key_offset(1, s));
            if (m >= a.heads) w = u32x4{0u, 0u, 0u, 0u};
            rest[s] = __builtin_bit_cast(bf16x8, w);
          }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) o[ht][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        top[ht] = kNone;
        l[ht] = 0.0f;
      }
    }
    const int tiles = steps_of<T>(p.end - p.begin);
    for (int t = 0; t < tiles; ++t, ++g) {
      // this tile is there (the first one came before the queries), and all waves are done with the one before or with the queries
      if (t == 0) lds_barrier();
      else loads_barrier();
      const char* tile = lds + (g & 1) * Sh::TILE;
      char* const to = lds + (~g & 1) * Sh::TILE;
      int asked = 0;
      // Loads of the next tile, `n` of them or what is left; behind the last one they bring rows that nobody reads.
      auto ask = [&](int n) {
#pragma unroll
        for (int i = 0; i < n; ++i)
          if (asked + i < Sh::LOADS) rows.load(to, asked + i, wave);
        asked += n;
      };
      constexpr int LEFT = Sh::LOADS - (KS + 1) / 2;           // not beside the scores: a quarter before them, half beside the weights, then the rest
      ask(LEFT / 4);
      const bool full = seen == RowTiles<Sh>::kFull;
      if (!full) {                     // a weight of zero does not take out a NaN or an infinity
        for (int i = threadIdx.x; i < T * NC; i += 64 * W) {
          const int row = i / NC;
          if ((row & 15) >= (int)(seen >> (8 * (row >> 4)) & 255)) *(u32x4*)(lds + (g & 1) * Sh::TILE + 16 * i) = u32x4{0u, 0u, 0u, 0u};
        }
        lds_barrier();
      }
      // reads ahead of the products that take them, in this order
      f32x4 s[HW][B];
      bf16x8 key[kKeysAhead + 1][B];
      auto read_keys = [&](int ks) {
#pragma unroll
        for (int i = 0; i < B; ++i)
          key[ks % (kKeysAhead + 1)][i] = *(const bf16x8*)(tile + 16 * Sh::ROW * B * part + key_at[ks % Sh::kKeyBases] + Sh::key_offset(i, ks));
      };
#pragma unroll
      for (int ks = 0; ks < kKeysAhead; ++ks) read_keys(ks);
#pragma unroll
      for (int ht = 0; ht < HW; ++ht)
#pragma unroll
        for (int i = 0; i < B; ++i) s[ht][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if (ks + kKeysAhead < KS) read_keys(ks + kKeysAhead);
        if (ks % 2 == 0) ask(1);
#pragma unroll
        for (int i = 0; i < B; ++i)
#pragma unroll
          for (int ht = 0; ht < HW; ++ht) s[ht][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(key[ks % (kKeysAhead + 1)][i], q[ht][ks], s[ht][i], 0, 0, 0);
        if constexpr (Sh::kQueryPairs)
          if (ks < R / 32)
#pragma unroll
            for (int i = 0; i < B; ++i) s[0][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(key[ks % (kKeysAhead + 1)][i], rest[ks], s[0][i], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      // this wave's weights, if no score is far above the maximum so far
      float high[HW];
      bool raised = false;
      auto weigh = [&](int ht) {
        const float at = top[ht] == kNone ? 0.0f : top[ht];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < B; ++i) {
          float e[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            e[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[ht][i][r], a.c, -at));
            sum += e[r];
          }
          weights[(N2 * ht * NB + part * B + i) * 64] = u32x2{f2_bf16(e[0], e[1]), f2_bf16(e[2], e[3])};
          if constexpr (N2 == 2) weights[((2 * ht + 1) * NB + part * B + i) * 64] = u32x2{f2_bf16(bf16_rest(e[0]), bf16_rest(e[1])), f2_bf16(bf16_rest(e[2]), bf16_rest(e[3]))};
        }
        return sum;
      };
      float sum[HW];
#pragma unroll
      for (int ht = 0; ht < HW; ++ht) {
        high[ht] = kNone;
#pragma unroll
        for (int i = 0; i < B; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (!full) s[ht][i][r] = 4 * quarter + r < (int)(seen >> (8 * (part * B + i)) & 255) ? s[ht][i][r] : kNone;
            high[ht] = fmaxf(high[ht], s[ht][i][r]);
          }
        high[ht] *= a.c;
        raised = raised || high[ht] > top[ht] + kSlack;
        sum[ht] = weigh(ht);
        ask(LEFT / 2 / HW);
      }
      const int raises = __any(raised) ? 1 : 0;
      if (lane == 0) flags[wave] = raises;
      lds_barrier();
      int any = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) any |= flags[i];
      if (__builtin_amdgcn_readfirstlane(any)) {     // the same for all waves: new maxima, and the weights again
#pragma unroll
        for (int ht = 0; ht < HW; ++ht) {
          const float most = quarters_max(high[ht]);
          if (quarter == 0) highs[(part * HW + ht) * 16] = most;
        }
        lds_barrier();                 // flags and weights have been read or are not needed, maxima are there
#pragma unroll
        for (int ht = 0; ht < HW; ++ht) {
          const float up = fmaxf(top[ht], fmaxf(highs[ht * 16], highs[(HW + ht) * 16])), f = top[ht] == kNone ? 0.0f : exp2f(top[ht] - up);
          top[ht] = up;
          l[ht] *= f;
#pragma unroll
          for (int j = 0; j < J; ++j) o[ht][j] *= f;
          sum[ht] = weigh(ht);
        }
        lds_barrier();
      }
      // C^T, 16 columns of two blocks
      constexpr int PAIRS = NB / 2, STEPS = PAIRS * J;
      u32x2 v[kValuesAhead + 1][2];
      auto read_values = [&](int n) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          v[n % (kValuesAhead + 1)][i] = read_turned(tile + value_at[n / PAIRS % Sh::kValueBases] + Sh::value_offset(2 * (n % PAIRS) + i, n / PAIRS));
      };
      bf16x8 w[HW][N2][PAIRS];
#pragma unroll
      for (int ht = 0; ht < HW; ++ht) {
        l[ht] += sum[ht];
#pragma unroll
        for (int k = 0; k < N2 * PAIRS; ++k) {
          const u32x2 x = weights[(N2 * ht * NB + 2 * k) * 64], y = weights[(N2 * ht * NB + 2 * k + 1) * 64];
          w[ht][k / PAIRS][k % PAIRS] = __builtin_bit_cast(bf16x8, u32x4{x[0], x[1], y[0], y[1]});
        }
      }
#pragma unroll
      for (int n = 0; n < kValuesAhead; ++n) read_values(n);
      constexpr int REST = LEFT - LEFT / 4 - LEFT / 2 / HW * HW, EVERY = REST ? STEPS / REST : STEPS;
#pragma unroll
      for (int n = 0; n < STEPS; ++n) {
        if (n + kValuesAhead < STEPS) read_values(n + kValuesAhead);
        if (REST && n % EVERY == 0) ask(1);
        const u32x2 x = v[n % (kValuesAhead + 1)][0], y = v[n % (kValuesAhead + 1)][1];
#pragma unroll
        for (int e = 0; e < N2; ++e)
#pragma unroll
          for (int ht = 0; ht < HW; ++ht)
            o[ht][n / PAIRS] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, u32x4{x[0], x[1], y[0], y[1]}), w[ht][e][n % PAIRS], o[ht][n / PAIRS], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      seen = coming;
      if (rows.more) {
        rows.step(a.split, lane);
        coming = rows.find_rows(a, wave);
      }
    }
    // both waves' sums of weights
#pragma unroll
    for (int ht = 0; ht < HW; ++ht) {
      l[ht] = quarters_sum(l[ht]);
      if (quarter == 0) highs[(part * HW + ht) * 16] = l[ht];
    }
    const int64_t place = p.place;
    const bool more = p.next(a.split, threadIdx.x);
    lds_barrier();
    if (more) ask_queries();
    asm volatile("" ::: "memory");    // no store goes before them: they are counted
    stored = tile16 + HW <= a.tiles;
#pragma unroll
    for (int ht = 0; ht < HW; ++ht) {
      if (tile16 + ht >= a.tiles) continue;
      const int head = 16 * (tile16 + ht) + m;
      const float all = highs[ht * 16] + highs[(HW + ht) * 16];
      // 1 KB a store; as rows of a head they would be 64 pieces of 8 bytes each, which took 17000 clocks
      float* to = a.part + ((place * a.tiles + tile16 + ht) * (R / 16) + J * part) * 256 + 4 * lane;
#pragma unroll
      for (int j = 0; j < J; ++j) *(f32x4*)(to + 256 * j) = o[ht][j];
      if (part == 0 && quarter == 0) {
        float* ml = a.ml + 2 * (place * a.tiles * 16 + head);
        ml[0] = top[ht] == kNone && all != 0.0f ? 0.0f : top[ht];            // scores of NaN alone: not "nothing seen"
        ml[1] = all;
      }
    }
    if (!more) break;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");             // LDS is not given up before the last loads have come
}

// Sum of a request's pieces for 16 heads, as join_kernel, from sums in the order of the instructions' results, written as rows of a head.
// Few pieces: a wave has 128 columns of all 16 heads, and the rows go out through LDS. Many pieces: a workgroup has 4 columns (256
// bytes of a piece), and 32 parts of 8 waves share the pieces, so that a request's megabytes come through many compute units at once
// (512 pieces of 16 heads and 512 columns: 32 workgroups 15.7 us, 128 of them 6).
template <int R, bool MANY>
struct LatentJoinShape {
  static constexpr int B = MANY ? 16 : 4;                      // pieces asked for at once
  static constexpr int WAVES = MANY ? 8 : R / 128, Z = MANY ? R / 4 : 1;
};
__device__ __forceinline__ void latent_lse(const LatentArgs& a, int b, int head, float top, float l) {
  a.lse[b * a.lse_b + head] = l == 0.0f ? kNone : (top + log2f(l)) / kLog2E;
}
template <int R, bool MANY>
__global__ __launch_bounds__((64 * LatentJoinShape<R, MANY>::WAVES)) void latent_join_kernel(LatentArgs a) {
  constexpr int B = LatentJoinShape<R, MANY>::B, JW = MANY ? 1 : 8, K = MANY ? 32 : 1;
  constexpr int W = MANY ? 8 : 1;
  __shared__ f32x4 red[W][16];
  __shared__ float tops[W][16], sums[W][16];
  __shared__ __attribute__((aligned(16))) uint16_t out[MANY ? 1 : 16][MANY ? 1 : 2 * R + 8];
  const int lane = threadIdx.x & 63, m = lane & 15, wave = threadIdx.x >> 6;
  const int b = blockIdx.y, tile16 = blockIdx.x, head = 16 * tile16 + m;
  const int quarter = MANY ? blockIdx.z & 3 : lane >> 4, k = MANY ? 4 * wave + (lane >> 4) : 0, j0 = MANY ? blockIdx.z >> 2 : 8 * wave;
  const int first = a.split.pieces[2 * b], n = a.split.pieces[2 * b + 1];
  float top = kNone, l = 0.0f;
  f32x4 o[JW];
#pragma unroll
  for (int j = 0; j < JW; ++j) o[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int i = k; i < n; i += K * B) {
    float pm[B], pl[B];
    f32x4 po[B][JW];
#pragma unroll
    for (int e = 0; e < B; ++e) {
      const int at = i + e * K;
      const int64_t row = (int64_t)(first + (at < n ? at : i)) * a.tiles + tile16;
      const float2 v = *(const float2*)(a.ml + 2 * (16 * row + m));
      pm[e] = at < n ? v.x : kNone;
      pl[e] = v.y;
#pragma unroll
      for (int j = 0; j < JW; ++j) po[e][j] = *(const f32x4*)(a.part + (row * (R / 16) + j0 + j) * 256 + 4 * (16 * quarter + m));
    }
    float t = top;
#pragma unroll
    for (int e = 0; e < B; ++e) t = pm[e] > t || pm[e] != pm[e] ? pm[e] : t;
    const float f = top == kNone ? 0.0f : exp2f(top - t);
    l *= f;
#pragma unroll
    for (int j = 0; j < JW; ++j) o[j] *= f;
#pragma unroll
    for (int e = 0; e < B; ++e) {
      if (pm[e] == kNone) continue;
      const float w = exp2f(pm[e] - t);
      l = __builtin_fmaf(w, pl[e], l);
#pragma unroll
      for (int j = 0; j < JW; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[j][r] = __builtin_fmaf(w, po[e][j][r], o[j][r]);
    }
    top = t;
  }
  if constexpr (MANY) {
    // the wave's four parts, then the waves, in order
    const float most = quarters_max(top), w4 = top == kNone ? 0.0f : exp2f(top - most);
    l = quarters_sum(top == kNone ? 0.0f : l * w4);
    f32x4 y;
#pragma unroll
    for (int r = 0; r < 4; ++r) y[r] = quarters_sum(top == kNone ? 0.0f : o[0][r] * w4);
    if (lane < 16) {
      tops[wave][m] = most;
      sums[wave][m] = l;
      red[wave][m] = y;
    }
    __syncthreads();
    if (threadIdx.x >= 16 || head >= a.heads) return;
    float t = kNone;
#pragma unroll
    for (int w = 0; w < W; ++w) t = tops[w][m] > t ? tops[w][m] : t;
    l = 0.0f;
    y = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (tops[w][m] == kNone) continue;
      const float f = exp2f(tops[w][m] - t);
      l = __builtin_fmaf(f, sums[w][m], l);
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = __builtin_fmaf(f, red[w][m][r], y[r]);
    }
    put_mean(a.mean + ((int64_t)b * a.heads + head) * (2 * R) + 16 * j0 + 4 * quarter, R, y * (l == 0.0f ? 0.0f : 1.0f / l));
    if (a.lse && blockIdx.z == 0) latent_lse(a, b, head, t, l);
  } else {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int j = 0; j < JW; ++j) put_mean(&out[m][16 * (j0 + j) + 4 * quarter], R, o[j] * inv);
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * R / 4; i += 64 * LatentJoinShape<R, MANY>::WAVES) {
      const int row = i / (R / 4), c = i % (R / 4);
      if (16 * tile16 + row < a.heads) *(u32x4*)(a.mean + ((int64_t)b * a.heads + 16 * tile16 + row) * (2 * R) + 8 * c) = *(const u32x4*)&out[row][8 * c];
    }
    if (a.lse && j0 == 0 && quarter == 0 && head < a.heads) latent_lse(a, b, head, top, l);
  }
}

// absorb_kernel: a[b][h][n] = bf16( sum_k x[b][h][k] w[h][k][n] ) and, for pairs, what the rounding left, the keys' weights on the query's side, written with the rope part
// behind them. The matrix has k rows of n, so a lane takes 8 k of 8 n and one byte permutation per pair of k and n
// turns them. A wave has 16 rows of x and 128 columns; the weights are read once per 16 rows.
struct AbsorbArgs {
  const char* x;
  const char* w;
  char* a;
  int64_t x_b, x_h, w_h;             // bytes
  int64_t rest;                      // bytes from a to what its rounding left, 0: not kept
  int32_t batch, heads, n, rope;     // n a multiple of 128
};

template <int K>
__global__ __launch_bounds__(64) void absorb_kernel(AbsorbArgs a) {
  const int lane = threadIdx.x, m = lane & 15, quarter = lane >> 4;
  const int h = blockIdx.y, b0 = 16 * blockIdx.z;
  const char* x = a.x + min(b0 + m, a.batch - 1) * a.x_b + h * a.x_h;
  const char* w = a.w + h * a.w_h;
  // chunk c of 8 columns of a row
  auto at = [&](int b, int c) { return a.a + 2 * ((int64_t)b * a.heads + h) * (a.n + a.rope) + 16 * c; };
  constexpr int N = 8;
  f32x4 acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int n0 = 128 * blockIdx.x;               // lane's columns n0 + 8 m + 0..7
  bf16x8 xv[K / 32];
  u32x4 r[K / 32][8];
#pragma unroll
  for (int k = 0; k < K / 32; ++k) {
    xv[k] = *(const bf16x8*)(x + 2 * (32 * k + 8 * quarter));
#pragma unroll
    for (int i = 0; i < 8; ++i) r[k][i] = *(const u32x4*)(w + 2 * ((int64_t)(32 * k + 8 * quarter + i) * a.n + n0 + 8 * m));
  }
  __builtin_amdgcn_sched_barrier(0);   // all loads before the first product
#pragma unroll
  for (int k = 0; k < K / 32; ++k)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      u32x4 v;
#pragma unroll
      for (int t = 0; t < 4; ++t) v[t] = __builtin_amdgcn_perm(r[k][2 * t + 1][j / 2], r[k][2 * t][j / 2], j % 2 ? 0x07060302u : 0x05040100u);
      acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[k], __builtin_bit_cast(bf16x8, v), acc[j], 0, 0, 0);
    }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = b0 + 4 * quarter + i;
    if (b >= a.batch) break;
    u32x4 v;
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = f2_bf16(acc[2 * t][i], acc[2 * t + 1][i]);
    *(u32x4*)at(b, n0 / 8 + m) = v;
    if (a.rest == 0) continue;
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = f2_bf16(bf16_rest(acc[2 * t][i]), bf16_rest(acc[2 * t + 1][i]));
    *(u32x4*)(at(b, n0 / 8 + m) + a.rest) = v;
  }
  if (blockIdx.x == 0) {
    const int chunks = a.rope / 8;
    for (int i = lane; i < 16 * chunks; i += 64) {
      const int b = b0 + i / chunks, c = i % chunks;
      if (b < a.batch) *(u32x4*)at(b, a.n / 8 + c) = *(const u32x4*)(a.x + b * a.x_b + h * a.x_h + 2 * (K + 8 * c));
    }
  }
}

// values_product_kernel: y[b][h][n] = bf16( sum_k (x_hi + x_lo)[b][h][k] w[h][n][k] ). A workgroup has one head: a wave 16 of its N columns, their
// weights in registers; rows of x come to LDS by direct loads, 16 requests at a time, two tiles in turn, once for all columns.
struct ValuesArgs {
  const char* x;                     // [batch][heads][2][K]
  const char* w;
  uint16_t* y;
  int64_t w_h;                       // bytes
  int64_t y_b, y_h;                  // elements
  int32_t batch, heads;
};

constexpr int kValueTiles = 2;       // tiles of 16 requests a workgroup has at most
constexpr int values_lds(int K) { return 2 * 16 * 4 * K; }
template <int K, int N>
__global__ __launch_bounds__(4 * N) void values_product_kernel(ValuesArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  constexpr int KS = K / 32, W = N / 16, NC = K / 8, PER = 64 / NC;      // chunks of a row; rows of 64 chunks
  const int lane = threadIdx.x & 63, m = lane & 15, quarter = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = blockIdx.x, b_tiles = (a.batch + 15) / 16, t0 = kValueTiles * blockIdx.y, t1 = min(b_tiles, t0 + kValueTiles);
  // chunk c of the rows 2 b, 2 b + 1 lies at c ^ (b & 15): the 16 rows of an operand on different banks
  auto load = [&](int tile) {
    char* to = lds + (tile & 1) * (64 * K);
    const int rows = 2 * min(16, a.batch - 16 * tile);
#pragma unroll
    for (int i = 0; i < 32 / PER / W; ++i) {
      const int r = PER * (i * W + wave), row = r + lane / NC, c = (lane % NC) ^ (row >> 1);
      if (r < rows)
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(a.x + (((int64_t)(16 * tile + (row >> 1)) * a.heads + h) * 2 + (row & 1)) * (2 * K) + 16 * c),
                                         (__attribute__((address_space(3))) void*)(to + r * (2 * K)), 16, 0, 0);
    }
  };
  load(t0);
  const char* w = a.w + h * a.w_h + (int64_t)(16 * wave + m) * (2 * K) + 16 * quarter;
  bf16x8 wv[KS];
#pragma unroll
  for (int k = 0; k < KS; ++k) wv[k] = *(const bf16x8*)(w + 64 * k);
  for (int tile = t0; tile < t1; ++tile) {
    loads_barrier();
    if (tile + 1 < t1) load(tile + 1);
    const char* x = lds + (tile & 1) * (64 * K) + 4 * K * m;             // rows behind the last request: whatever lies there, and not stored
    f32x4 acc[2] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(*(const bf16x8*)(x + 2 * K * i + 16 * ((4 * k + quarter) ^ m)), wv[k], acc[i], 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = 16 * tile + 4 * quarter + i;
      if (b < a.batch) a.y[b * a.y_b + h * a.y_h + 16 * wave + m] = f_bf16(acc[0][i] + acc[1][i]);
    }
  }
}

}  // namespace ops
}  // namespace fg
