// Latent attention, expanded form, of ragged prompts: keys [W_k c | r] and values
// W_v c of every head are formed once (expand_kernel), then
//   out[i][h] = sum_j w_ij v_j,  w = softmax over j <= nk - nq + i of scale (q_nope . k_j + q_rope . r_j)
// (prompt_kernel), 2 H (2 M + P) flops a pair: matrix instructions bound it.
//
// prompt_kernel: a workgroup has W waves of 32 queries of one head; tiles of 64
// keys and values go through LDS by direct loads, two in turn. Both products are
// 32x32x16 instructions with the query in the lane:
//   S^T[key][query] = K Q^T;   O^T[dim][query] += V^T P^T
// Lane l holds of S^T the keys 8 a + 4 (l / 32) + 0..3, which two at a time are a legal
// order of the 16 keys of a second product, whose V^T comes by transposing reads of 4 keys; so
// a query's weights, maximum and sum stay in its lane.
// The rope part of the keys is read from the latent rows as it is; heads share it.
// Keys that a query does not see have weight zero, but zero times a NaN or an infinity of their
// values is NaN: in tiles where some are hidden, keys with such values are multiplied one by one, and only into
// the queries that see them.
#pragma once

#include "fg_latent.hpp"

namespace fg {
namespace ops {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// ------------------------------------------------------------------- expand
// kv[t][n] = bf16( sum_r lat[t][r] w[n][r] ), n over heads and their 2 M rows: 128 x 128 tiles, four waves of 64 x 64, 32 r at a time through LDS
// by direct loads, four stages in turn, of which three are in flight (with two stages of 64 and one in flight 16384 x 4096 x 512 took 118 us).
struct ExpandArgs {
  const char* lat;
  const char* w;
  uint16_t* kv;
  int64_t ld;                        // bytes of a latent row
  int64_t rows;
  int32_t n, r;                      // n = heads * 2 M, any multiple of 128
};

constexpr int kExpandTile = 128, kExpandStages = 4, kExpandStage = 2 * kExpandTile * 64;
__global__ __launch_bounds__(256, 2) void expand_kernel(ExpandArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63, l32 = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = kExpandTile * blockIdx.x, wm = wave >> 1, wn = wave & 1;
  const int64_t t0 = (int64_t)kExpandTile * blockIdx.y;
  const int left = (int)min((int64_t)kExpandTile, a.rows - t0) - 1;
  // 16 rows of 64 bytes a load, two loads of each operand a wave; chunks permuted by the row's group of four, so that 16 rows differ in banks
  const char* const lat = a.lat + t0 * a.ld;
  const char* const w = a.w + 2 * (int64_t)n0 * a.r;
  uint32_t at[2], wt[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 16 * (2 * wave + i) + (lane >> 2), c = (lane & 3) ^ ((row >> 2) & 3);
    at[i] = (uint32_t)min(row, left) * (uint32_t)a.ld + 16 * c;
    wt[i] = 2 * (uint32_t)row * (uint32_t)a.r + 16 * c;
  }
  auto load = [&](int s) {
    char* to = lds + s % kExpandStages * kExpandStage + 1024 * (2 * wave);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      load_to_lds(lat + 64 * s, at[i], to + 1024 * i);
      load_to_lds(w + 64 * s, wt[i], to + kExpandStage / 2 + 1024 * i);
    }
  };
  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  const int steps = a.r / 32;          // at least 8
  load(0);
  load(1);
  load(2);
  for (int s = 0; s < steps; ++s) {
    // a wave has four loads a stage: those of the two later stages may be under way
    if (s + 2 < steps) asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
    else if (s + 1 < steps) asm volatile("s_waitcnt vmcnt(4)" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    lds_barrier();
    if (s + 3 < steps) load(s + 3);
    const char* x = lds + s % kExpandStages * kExpandStage;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      bf16x8 u[2], v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int ru = 64 * wn + 32 * i + l32, rv = 64 * wm + 32 * i + l32;
        u[i] = *(const bf16x8*)(x + kExpandStage / 2 + ru * 64 + 16 * ((2 * k + half) ^ ((ru >> 2) & 3)));
        v[i] = *(const bf16x8*)(x + rv * 64 + 16 * ((2 * k + half) ^ ((rv >> 2) & 3)));
      }
      // rows of the result are columns n: a lane has 4 consecutive ones of a token
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(u[j], v[i], acc[i][j], 0, 0, 0);
    }
  }
  // rows of 256 bytes go out through LDS: stored from the registers they would be pieces of 8 bytes, which take as long as the products
  constexpr int OUT = 2 * kExpandTile + 16;
  static_assert(kExpandTile * OUT <= kExpandStages * kExpandStage, "the tile fits the stages");
  lds_barrier();
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *(u32x2*)(lds + (64 * wm + 32 * i + l32) * OUT + 2 * (64 * wn + 32 * j + 2 * e + 4 * half)) =
            u32x2{f2_bf16(acc[i][j][e], acc[i][j][e + 1]), f2_bf16(acc[i][j][e + 2], acc[i][j][e + 3])};
  lds_barrier();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = 16 * i + (threadIdx.x >> 4), c = threadIdx.x & 15;
    if (row <= left) *(u32x4*)(a.kv + (t0 + row) * a.n + n0 + 8 * c) = *(const u32x4*)(lds + row * OUT + 16 * c);
  }
}

// ------------------------------------------------------------------- prompt
struct PromptArgs {
  const char* q;
  const char* kv;                    // bf16 [keys][heads][2 M]
  const char* lat;                   // latent rows, for their rope part
  uint16_t* out;
  float* lse;
  const int32_t* q_starts;
  const int32_t* k_starts;
  int64_t q_t, q_h, ld;              // bytes
  int64_t out_t, out_h, lse_t;       // elements
  int64_t q_rows, k_rows;
  int32_t batch, heads, r, items;    // items: workgroups a head
  float c;
};

// In LDS: 64 rows of keys' nope part, of their rope part and of values, 4, 8 or 16 chunks of 16 bytes each.
template <int M, int P>
struct PromptShape {
  static constexpr int KC = M / 8, RC = P / 8;
  static constexpr int KB = 1024 * KC, KEYS = KB + 1024 * RC, STAGE = KEYS + KB;
  // 16 rows of one chunk on different banks
  template <int N>
  static __device__ __forceinline__ int key_place(int c, int t) {
    return c ^ (N == 16 ? t & 15 : N == 8 ? (t >> 1) & 7 : (t >> 2) & 3);
  }
  // 32 dims of 4 rows on different banks
  static __device__ __forceinline__ int value_place(int c, int t) { return c ^ (KC == 16 ? (t & 3) << 2 : (t & 2) << 1); }
};

// Starts lie within the rows: one outside counts as the nearest. So all requests together have no more tiles than there are items.
__device__ __forceinline__ int start_of(const int32_t* starts, int i, int64_t rows) { return min(max(starts[i], 0), (int)rows); }

// Request and tile of Q queries of item `item` (in request order); false if there are fewer.
template <int T, int Q>
__device__ __forceinline__ bool find_queries(const PromptArgs& a, int item, SplitShared& sh, int& b, int& tile) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (a.batch + T - 1) / T, from = min(tid * per, a.batch), to = min(from + per, a.batch);
  auto tiles = [&](int i) { return max(0, start_of(a.q_starts, i + 1, a.q_rows) - start_of(a.q_starts, i, a.q_rows) + Q - 1) / Q; };
  int count = 0;
  for (int i = from; i < to; ++i) count += tiles(i);
  int upto = lanes_before_and_own(count);
  if (lane == 63) sh.sum[wave] = upto;
  if (tid == 0) sh.found[0] = -1;
  __syncthreads();
  for (int w = 0; w < wave; ++w) upto += sh.sum[w];
  if (item < upto && item >= upto - count) {
    int at = upto - count;
    for (int i = from; i < to; ++i) {
      const int n = tiles(i);
      if (item < at + n) {
        sh.found[0] = i;
        sh.found[1] = item - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  b = __builtin_amdgcn_readfirstlane(sh.found[0]);
  tile = __builtin_amdgcn_readfirstlane(sh.found[1]);
  return b >= 0;
}

template <int M, int P, int W>
__global__ __launch_bounds__(64 * W, 2) void prompt_kernel(PromptArgs a) {
  typedef PromptShape<M, P> Sh;
  constexpr int KC = Sh::KC, RC = Sh::RC, KS = (M + P) / 16, DT = M / 32;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ SplitShared sh;
  const int lane = threadIdx.x & 63, l32 = lane & 31, half = lane >> 5, m = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // workgroups go round the 8 dies; a die takes neighbouring items, which share a head's keys, in its L2
  const uint32_t share = gridDim.x * gridDim.y / 8, at_grid = blockIdx.y * gridDim.x + blockIdx.x;
  const int id = (int)((at_grid & 7) * share + (at_grid >> 3));
  if ((uint32_t)id >= (uint32_t)a.items * (uint32_t)a.heads) return;
  const int h = id / a.items;
  int b, tile;
  // last tiles first: they see the most keys
  if (!find_queries<64 * W, 32 * W>(a, a.items - 1 - (id - h * a.items), sh, b, tile)) return;
  const int q_first = start_of(a.q_starts, b, a.q_rows), nq = start_of(a.q_starts, b + 1, a.q_rows) - q_first;
  const int k_first = start_of(a.k_starts, b, a.k_rows), nk = start_of(a.k_starts, b + 1, a.k_rows) - k_first;
  const int i0 = 32 * W * tile, i = i0 + 32 * wave + l32;          // this lane's query
  const int last = i < nq ? nk - nq + i : -1;                      // the last key that it sees
  const int wave_first = nk - nq + i0 + 32 * wave;                 // what the wave's first query sees
  const int wave_last = min(wave_first + 31, nk - 1);
  const int keys = min(nk, nk - nq + min(i0 + 32 * W, nq)), tiles = keys <= 0 ? 0 : (keys + 63) / 64;

  bf16x8 q[KS];
  const char* qrow = a.q + (int64_t)(q_first + min(i, nq - 1)) * a.q_t + h * a.q_h;
#pragma unroll
  for (int s = 0; s < KS; ++s) q[s] = *(const bf16x8*)(qrow + 2 * (16 * s + 8 * half));
  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = 0.0f;
  float top = kNone, l = 0.0f;

  const uint32_t kv_row = (uint32_t)a.heads * 4 * M;
  const char* kv = a.kv + (int64_t)k_first * kv_row + h * (4 * M);
  const char* rope = a.lat + (int64_t)k_first * a.ld + 2 * a.r;
  // a wave's loads of one area: N chunks of 64 rows, `row` bytes apart from `base` on; rows behind the last key are it again
  auto area = [&](auto chunks, const char* base, uint32_t pitch, int left, char* to, auto place) {
    constexpr int N = decltype(chunks)::value;
#pragma unroll
    for (int n = 0; n < (N + W - 1) / W; ++n) {
      if (N % W != 0 && n * W + wave >= N) break;
      const int slot = (n * W + wave) * 64 + lane, row = slot / N, c = place(slot % N, row);
      load_to_lds(base, (uint32_t)min(row, left) * pitch + 16 * c, to + (n * W + wave) * 1024);
    }
  };
  auto load = [&](int t) {
    char* to = lds + (t & 1) * Sh::STAGE;
    const int left = nk - 1 - 64 * t;
    const char* rows = kv + 64 * (int64_t)t * kv_row;
    area(std::integral_constant<int, KC>(), rows, kv_row, left, to, [](int c, int r) { return Sh::template key_place<KC>(c, r); });
    area(std::integral_constant<int, RC>(), rope + 64 * (int64_t)t * a.ld, (uint32_t)a.ld, left, to + Sh::KB,
         [](int c, int r) { return Sh::template key_place<RC>(c, r); });
    area(std::integral_constant<int, KC>(), rows + 2 * M, kv_row, left, to + Sh::KEYS, [](int c, int r) { return Sh::value_place(c, r); });
  };
  if (tiles > 0) load(0);
  bf16x8 w[4];                         // rounded weights; as pairs 16384 tokens took 2.4 ms instead of 1.5
  // Values of tile t: 16 keys (k) and 32 dims (d) at a time, keys 16 k + 4 half + 0..3 and 8 more, dims 32 d + lane % 32
  const int vrow = 4 * half + (m >> 2), vc = 2 * ((lane >> 4) & 1) + ((m & 3) >> 1);
  auto value = [&](const char* vt, int n) {
    const int k = n / DT, d = n % DT;
    const char* from = vt + (16 * k + vrow) * (16 * KC) + 16 * Sh::value_place(4 * d + vc, vrow) + 8 * (m & 1);
    const u32x2 x = read_turned(from), y = read_turned(from + 8 * (16 * KC));
    return u32x4{x[0], x[1], y[0], y[1]};
  };
  auto add_values = [&](int t) {
    const char* vt = lds + (t & 1) * Sh::STAGE + Sh::KEYS;
    if (64 * t + 63 <= wave_first && 64 * t + 64 <= nk) {
      constexpr int N = 4 * DT, AHEAD = 3;
      u32x4 v[AHEAD + 1];
#pragma unroll
      for (int n = 0; n < AHEAD; ++n) v[n] = value(vt, n);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if (n + AHEAD < N) v[(n + AHEAD) % (AHEAD + 1)] = value(vt, n + AHEAD);
        o[n % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v[n % (AHEAD + 1)]), w[n / DT], o[n % DT], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      return;
    }
#pragma unroll
    for (int n = 0; n < 4 * DT; ++n) {
      const int k = n / DT, d = n % DT;
      const u32x4 v = value(vt, n);
      bool odd = false;
#pragma unroll
      for (int j = 0; j < 4; ++j) odd = odd || (v[j] & 0x7f80u) == 0x7f80u || (v[j] & 0x7f800000u) == 0x7f800000u;
      if (!__any(odd)) {
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v), w[k], o[d], 0, 0, 0);
        continue;
      }
      // one key at a time, kept by the queries that see it
#pragma unroll 1
      for (int j = 0; j < 8; ++j)
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {
          u32x4 one, pw;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t mask = half == g && e == j / 2 ? (j & 1 ? 0xffff0000u : 0xffffu) : 0u;
            one[e] = v[e] & mask;
            pw[e] = __builtin_bit_cast(u32x4, w[k])[e] & mask;
          }
          const f32x16 sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, one), __builtin_bit_cast(bf16x8, pw), o[d], 0, 0, 0);
          const int key = 64 * t + 16 * k + 4 * g + j % 4 + 8 * (j / 4);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[d][e] = key <= last ? sum[e] : o[d][e];
        }
    }
  };
  // A round adds the values of the tile before, then forms the scores and weights of the next one (in the other order the compiler's registers do
  // not suffice).
  int held = -1;                       // tile whose weights wait for their values, or none
  for (int t = 0; t <= tiles; ++t) {
    if (held >= 0) add_values(held);
    held = -1;
    if (t == tiles) break;
    loads_barrier();                   // tile t is there, and all waves are done with tile t - 1
    if (t + 1 < tiles) load(t + 1);
    if (64 * t > wave_last) continue;  // no query of this wave sees any of it
    held = t;
    const char* kt = lds + (t & 1) * Sh::STAGE;
    f32x16 s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[u][e] = 0.0f;
    constexpr int AHEAD = 2;
    bf16x8 key[AHEAD + 1][2];
    auto read_keys = [&](int ks) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = 32 * u + l32, c = 2 * ks + half;
        key[ks % (AHEAD + 1)][u] = *(const bf16x8*)(ks < M / 16 ? kt + row * (16 * KC) + 16 * Sh::template key_place<KC>(c, row)
                                                               : kt + Sh::KB + row * (16 * RC) + 16 * Sh::template key_place<RC>(c - KC, row));
      }
    };
#pragma unroll
    for (int ks = 0; ks < AHEAD; ++ks) read_keys(ks);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if (ks + AHEAD < KS) read_keys(ks + AHEAD);
#pragma unroll
      for (int u = 0; u < 2; ++u) s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(key[ks % (AHEAD + 1)][u], q[ks], s[u], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (64 * t + 63 > wave_first || 64 * t + 64 > nk) {      // some query of the wave does not see all of it
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int key_at = 64 * t + 32 * u + 8 * (e / 4) + 4 * half + e % 4;
          s[u][e] = key_at <= last ? s[u][e] : kNone;
        }
    }
    float high = kNone;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 16; ++e) high = fmaxf(high, s[u][e]);
    high *= a.c;
    if (__any(high > top + kSlack)) {
      const uint32_t hw = __float_as_uint(high);
      const auto x = __builtin_amdgcn_permlane32_swap(hw, hw, false, false);
      const float up = fmaxf(top, fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1])));
      const float f = top == kNone ? 0.0f : exp2f(top - up);
      top = up;
      l *= f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] *= f;
    }
    const float at = top == kNone ? 0.0f : top;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      u32x4 pk;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k / 2][8 * (k & 1) + e], a.c, -at));
        const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k / 2][8 * (k & 1) + e + 1], a.c, -at));
        l += x + y;
        pk[e / 2] = f2_bf16(x, y);
      }
      w[k] = __builtin_bit_cast(bf16x8, pk);
    }
  }
  const uint32_t lw = __float_as_uint(l);
  const auto x = __builtin_amdgcn_permlane32_swap(lw, lw, false, false);
  const float all = __uint_as_float(x[0]) + __uint_as_float(x[1]);
  const float inv = all == 0.0f ? 0.0f : 1.0f / all;
  // rows of 2 M bytes go out through LDS, a wave's own 32 at a time
  constexpr int OUT = 2 * M + 16;
  static_assert(32 * W * OUT <= 2 * Sh::STAGE, "the rows fit the stages");
  lds_barrier();                       // all waves are done with the last tile
  char* const rows_out = lds + wave * (32 * OUT);
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int e = 0; e < 16; e += 4)
      *(u32x2*)(rows_out + l32 * OUT + 2 * (32 * d + 2 * e + 4 * half)) = u32x2{f2_bf16(o[d][e] * inv, o[d][e + 1] * inv), f2_bf16(o[d][e + 2] * inv, o[d][e + 3] * inv)};
  uint16_t* const to = a.out + h * a.out_h;
#pragma unroll
  for (int n = 0; n < KC / 2; ++n) {
    const int slot = 64 * n + lane, row = slot / KC, c = slot % KC, qi = i0 + 32 * wave + row;
    const u32x4 v = *(const u32x4*)(rows_out + row * OUT + 16 * c);
    if (qi >= nq) continue;
    u32x2* at = (u32x2*)(to + (int64_t)(q_first + qi) * a.out_t + 8 * c);       // rows start on 8-byte boundaries
    at[0] = u32x2{v[0], v[1]};
    at[1] = u32x2{v[2], v[3]};
  }
  if (i >= nq) return;
  if (a.lse && half == 0)
    a.lse[(int64_t)(q_first + i) * a.lse_t + h] = all == 0.0f ? kNone : ((top == kNone ? 0.0f : top) + log2f(all)) / kLog2E;
}

}  // namespace ops
}  // namespace fg
