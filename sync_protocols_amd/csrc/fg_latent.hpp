// Latent attention, absorbed form, of one new token over a paged cache of rows
// [latent of R | rope of P], one for all heads:
//   a[b][h] = W_k[h]^T q_nope[b][h]                         heads_product, R columns
//   u[b][h] = sum_t w_t c_t,  w = softmax of scale (a . c_t + q_rope . r_t)       latent_kernel
//   out[b][h] = W_v[h] u[b][h]                              heads_product, M columns
// Keys and values are the same rows, so a row is read once, for up to 128 heads:
// 2 H (2 R + P) flops for 2 (R + P) bytes, 242 a byte with 128 heads of 512 + 64, near the ratio of the matrix to the memory rate.
//
// latent_kernel: tiles of 64 rows go to LDS by direct loads, two tiles in turn,
// and serve both products as 16x16x32 matrix instructions with the head in the lane:
//   S^T[token][head] = C A^T       C: 16 bytes of a row
//   U^T[dim][head] += C^T W^T      C^T by transposing reads: 4 tokens of a dim in a lane,
//                                  the tokens of the lane's own scores, so weights stay in the lane
// A wave owns 16 heads (all of A in registers) and with S = 1 all their columns.
// Fewer heads than 64 a workgroup leave waves free: then S of them share 16 heads, each
// takes 64 / S rows of the scores and R / S columns of the sum, and the scores of
// all 64 rows meet in LDS.
// Chunks of 16 bytes lie permuted in a row, so that the 16 rows of a key read and
// the 8 rows of a transposing read fall on different banks.
#pragma once

#include "fg_paged.hpp"

namespace fg {
namespace ops {

struct LatentArgs {
  SplitArgs split;
  const char* a;                     // bf16 [batch][heads][R]: the absorbed queries
  const char* q;                     // rope part of the queries
  const char* cache;
  uint16_t* out;                     // bf16 [batch][heads][2][R]: the mean, and what its rounding leaves
  float* lse;
  float* part;
  float* ml;
  int64_t q_b, q_h;                  // bytes
  int64_t c_page, lse_b;             // bytes, elements
  int32_t c_tok, heads;
  float c;
};

constexpr int kLatentTile = 64;
constexpr int kBlockTable = 512;                // blocks of 16 rows whose places are in LDS at a time
constexpr int kBlocksPerTile = kLatentTile / 16;

template <int R, int P, int HT, int S>
struct LatentShape {
  static constexpr int W = HT * S;              // waves
  static constexpr int NC = (R + P) / 8;        // chunks of a row
  static constexpr int KS = (R + P) / 32;       // matrix instructions of a score
  static constexpr int ROW = 2 * (R + P);
  static constexpr int TILE = kLatentTile * ROW;
  static constexpr int LDS_SCORES = 2 * TILE;
  static constexpr int SCORE_LD = kLatentTile + 4;
  static constexpr int LDS_TABLE = LDS_SCORES + (S > 1 ? HT * 16 * SCORE_LD * 4 : 0);
  static constexpr int LDS = LDS_TABLE + 8 * kBlockTable;
  static_assert(NC % 16 == 8 || NC % 16 == 4, "row");
  // Place of chunk c in row t. A row is 8 (or 4) chunks past a multiple of 16, 256 bytes, so rows of one parity (of one t % 4) share a half
  // (a quarter) of the banks.
  static __device__ __forceinline__ int place(int c, int t) {
    if constexpr (NC % 16 == 8) return c ^ ((((t >> 1) & 3) << 1) | ((t >> 3) & 1));
    else return c ^ ((((t >> 2) & 1) << 1) | ((t >> 3) & 1));
  }
};

template <int R, int P, int HT, int S>
__global__ __launch_bounds__(64 * HT * S, HT * S == 8 ? 2 : 1) void latent_kernel(LatentArgs a) {
  typedef LatentShape<R, P, HT, S> Sh;
  constexpr int W = Sh::W, KS = Sh::KS, NC = Sh::NC, J = R / S / 16;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ SplitShared sh;
  Piece p;
  if (!find_piece<64 * W, kLatentTile>(a.split, blockIdx.x, sh, p)) return;
  const int lane = threadIdx.x & 63, m = lane & 15, quarter = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ht = wave / S, part = wave % S;
  const int head = 16 * (HT * blockIdx.y + ht) + m;
  int64_t* table = (int64_t*)(lds + Sh::LDS_TABLE);
  float* scores = (float*)(lds + Sh::LDS_SCORES) + (ht * 16 + m) * Sh::SCORE_LD;
  const int block0 = p.begin / 16, tiles = (p.end - p.begin + kLatentTile - 1) / kLatentTile;

  bf16x8 q[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const int64_t row = (int64_t)p.b * a.heads + min(head, a.heads - 1);
    const char* from = s < R / 32 ? a.a + 2 * (row * R + 32 * s + 8 * quarter)
                                  : a.q + p.b * a.q_b + min(head, a.heads - 1) * a.q_h + 2 * (32 * s - R + 8 * quarter);
    u32x4 w = *(const u32x4*)from;
    if (head >= a.heads) w = u32x4{0u, 0u, 0u, 0u};
    q[s] = __builtin_bit_cast(bf16x8, w);
  }
  f32x4 o[J];
#pragma unroll
  for (int j = 0; j < J; ++j) o[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float top = kNone, l = 0.0f;

  // places of the blocks from tile t on, -1 for those without rows
  auto fetch = [&](int t) {
    for (int i = threadIdx.x; i < kBlockTable; i += 64 * W) {
      const int64_t tok = 16 * ((int64_t)block0 + kBlocksPerTile * t + i);
      int64_t at = -1;
      if (tok < p.len) {
        const int32_t pg = (int32_t)(tok / a.split.page), id = a.split.table[p.b * a.split.ldt + pg];
        if (id >= 0 && id < a.split.n_pages) at = id * a.c_page + (tok - (int64_t)pg * a.split.page) * a.c_tok;
      }
      table[i] = at;
    }
    __syncthreads();
  };
  constexpr int kTilesInTable = kBlockTable / kBlocksPerTile;
  auto load = [&](int t) {
    char* to = lds + (t & 1) * Sh::TILE;
    const int64_t* place = table + kBlocksPerTile * (t % kTilesInTable);
#pragma unroll
    for (int i = 0; i < (NC + W - 1) / W; ++i) {
      if (NC % W != 0 && i * W + wave >= NC) break;
      const int slot = (i * W + wave) * 64 + lane, row = slot / NC, c = Sh::place(slot - row * NC, row);
      const int64_t at = place[row >> 4];
      const char* from = a.cache + (at < 0 ? 0 : at + (row & 15) * (int64_t)a.c_tok) + 16 * c;
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                       (__attribute__((address_space(3))) void*)(to + (i * W + wave) * 1024), 16, 0, 0);
    }
  };
  if (tiles > 0) {
    fetch(0);
    load(0);
  }
  for (int t = 0; t < tiles; ++t) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();                   // tile t is there, and all waves are done with tile t - 1
    const char* tile = lds + (t & 1) * Sh::TILE;
    const int64_t* place = table + kBlocksPerTile * (t % kTilesInTable);
    const int tok0 = p.begin + kLatentTile * t, left = p.len - tok0;
    int seen[4];                       // rows of each block
    bool full = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      seen[i] = __builtin_amdgcn_readfirstlane(place[i] < 0 ? 0 : min(16, left - 16 * i));
      full = full && seen[i] == 16;
    }
    if (!full) {                       // a weight of zero does not take out a NaN or an infinity
      for (int i = threadIdx.x; i < kLatentTile * NC; i += 64 * W) {
        const int row = i / NC;
        if ((row & 15) >= seen[row >> 4]) *(u32x4*)(lds + (t & 1) * Sh::TILE + 16 * i) = u32x4{0u, 0u, 0u, 0u};
      }
      __syncthreads();
    }
    if (t + 1 < tiles) {
      if ((t + 1) % kTilesInTable == 0) {
        __syncthreads();               // place[] has been read
        fetch(t + 1);
      }
      load(t + 1);
    }
    f32x4 s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int B = 4 / S;           // this wave's blocks
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int row = 16 * (part * B + i) + m;
        const bf16x8 key = *(const bf16x8*)(tile + row * Sh::ROW + 16 * Sh::place(4 * ks + quarter, m));
        s[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(key, q[ks], s[i], 0, 0, 0);
      }
    if constexpr (S > 1) {
#pragma unroll
      for (int i = 0; i < B; ++i) *(f32x4*)(scores + 16 * (part * B + i) + 4 * quarter) = s[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = *(const f32x4*)(scores + 16 * i + 4 * quarter);
    }
    float high = kNone;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s[i][r] *= a.c;
        if (!full) s[i][r] = 4 * quarter + r < seen[i] ? s[i][r] : kNone;
        high = fmaxf(high, s[i][r]);
      }
    if (__any(high > top + kSlack)) {
      const float up = fmaxf(top, quarters_max(high)), f = top == kNone ? 0.0f : exp2f(top - up);
      top = up;
      l *= f;
#pragma unroll
      for (int j = 0; j < J; ++j) o[j] *= f;
    }
    const float at = top == kNone ? 0.0f : top;
    bf16x8 w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      u32x4 pk;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float e[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          e[r] = __builtin_amdgcn_exp2f(s[2 * k + i][r] - at);
          l += e[r];
        }
        pk[2 * i] = f2_bf16(e[0], e[1]);
        pk[2 * i + 1] = f2_bf16(e[2], e[3]);
      }
      w[k] = __builtin_bit_cast(bf16x8, pk);
    }
    // transposing read: lane m asks for dims 4 (m % 4) + 0..3 of row m / 4 and gets rows 0..3 of dim m
    const int row = 4 * quarter + (m >> 2);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = R / S / 8 * part + 2 * j + ((m & 3) >> 1);
      const char* from = tile + row * Sh::ROW + 16 * Sh::place(c, row) + 8 * (m & 1);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(from + 32 * k * Sh::ROW)));
        const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(from + (32 * k + 16) * Sh::ROW)));
        const bf16x8 v = __builtin_bit_cast(bf16x8, u32x4{x[0], x[1], y[0], y[1]});
        o[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, w[k], o[j], 0, 0, 0);
      }
    }
  }
  const float all = quarters_sum(l);
  if (head >= a.heads) return;
  const bool last = p.count == 1;
  const float inv = !last ? 1.0f : all == 0.0f ? 0.0f : 1.0f / all;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int d = R / S * part + 16 * j + 4 * quarter;
    if (last) {
      const f32x4 y = o[j] * inv;
      uint16_t* to = a.out + ((int64_t)p.b * a.heads + head) * (2 * R) + d;
      *(u32x2*)to = u32x2{f2_bf16(y[0], y[1]), f2_bf16(y[2], y[3])};
      *(u32x2*)(to + R) = u32x2{f2_bf16(bf16_rest(y[0]), bf16_rest(y[1])), f2_bf16(bf16_rest(y[2]), bf16_rest(y[3]))};
    } else {
      *(f32x4*)(a.part + ((int64_t)p.item * a.heads + head) * R + d) = o[j];
    }
  }
  if (part == 0 && quarter == 0) {
    const float t = top == kNone && all != 0.0f ? 0.0f : top;     // scores of NaN alone: not "nothing seen"
    if (last) {
      if (a.lse) a.lse[p.b * a.lse_b + head] = all == 0.0f ? kNone : (t + log2f(all)) / kLog2E;
    } else {
      float* to = a.ml + 2 * ((int64_t)p.item * a.heads + head);
      to[0] = t;
      to[1] = all;
    }
  }
}

// Products of every head's rows with its own matrix, few rows a head:
//   y[b][h][n] = bf16( sum_k x[b][h][k] w[h](k, n) )
// KN: the matrix has k rows of N (absorbing the keys' weights, transposed in registers: a lane takes 8 k of 8 n and
// one byte permutation per pair of k and n turns them); else n rows of K, as stored, and x has two numbers for each, K apart:
// the weighted mean as one bf16 would add an error as large as the result's own rounding.
// A wave has 16 rows of x and 128 (KN) or 16 columns; the weights are read once per 16 rows.
struct HeadsArgs {
  const char* x;
  const char* w;
  uint16_t* y;
  int64_t x_b, x_h, w_h;             // bytes
  int64_t y_b, y_h;                  // elements
  int32_t batch, heads, k, n;        // k a multiple of 32, n of 128 (KN), or of 64 and 16
};

template <bool KN>
__global__ __launch_bounds__(64) void heads_product_kernel(HeadsArgs a) {
  const int lane = threadIdx.x, m = lane & 15, quarter = lane >> 4;
  const int h = blockIdx.y, b0 = 16 * blockIdx.z;
  const char* x = a.x + min(b0 + m, a.batch - 1) * a.x_b + h * a.x_h;
  const char* w = a.w + h * a.w_h;
  if constexpr (KN) {
    constexpr int N = 8;
    f32x4 acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int n0 = 128 * blockIdx.x;             // lane's columns n0 + 8 m + 0..7
    for (int k = 0; k < a.k; k += 32) {
      const bf16x8 xv = *(const bf16x8*)(x + 2 * (k + 8 * quarter));
      u32x4 r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = *(const u32x4*)(w + 2 * ((int64_t)(k + 8 * quarter + i) * a.n + n0 + 8 * m));
#pragma unroll
      for (int j = 0; j < N; ++j) {
        u32x4 v;
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] = __builtin_amdgcn_perm(r[2 * t + 1][j / 2], r[2 * t][j / 2], j % 2 ? 0x07060302u : 0x05040100u);
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, __builtin_bit_cast(bf16x8, v), acc[j], 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = b0 + 4 * quarter + i;
      if (b >= a.batch) break;
      u32x4 v;
#pragma unroll
      for (int t = 0; t < 4; ++t) v[t] = f2_bf16(acc[2 * t][i], acc[2 * t + 1][i]);
      *(u32x4*)(a.y + b * a.y_b + h * a.y_h + n0 + 8 * m) = v;
    }
  } else {
    f32x4 acc[2] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
    const int n0 = 16 * blockIdx.x;
    const char* row = w + 2 * (int64_t)(n0 + m) * a.k;
#pragma unroll 4
    for (int k = 0; k < a.k; k += 64)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = 2 * (k + 32 * i + 8 * quarter);
        const bf16x8 wv = *(const bf16x8*)(row + at);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(*(const bf16x8*)(x + at), wv, acc[i], 0, 0, 0);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(*(const bf16x8*)(x + 2 * a.k + at), wv, acc[i], 0, 0, 0);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = b0 + 4 * quarter + i;
      if (b < a.batch) a.y[b * a.y_b + h * a.y_h + n0 + m] = f_bf16(acc[0][i] + acc[1][i]);
    }
  }
}

}  // namespace ops
}  // namespace fg
