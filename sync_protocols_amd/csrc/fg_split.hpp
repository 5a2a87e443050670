// Work of attention over a paged cache, split over the cache's length.
//
// The lengths are on the GPU, so the split is made there: a request's tokens are cut
// into pieces of about (all tokens) / target, at least `least` units of U tokens,
// and item i of the grid is the i-th piece of all requests. Every workgroup finds its
// own from the lengths by two sums over them, which takes less than a launch. A
// request without tokens has one empty piece, so that its outputs are written too.
// Pieces of one request that has several leave their sums (running maximum, sum of
// weights, weighted sum) in the workspace, and join_kernel adds them up in order.
#pragma once

#include "fg_ops.hpp"

namespace fg {
namespace ops {

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kNone = -__builtin_inff();
// The running maximum is only raised when a score exceeds it by more than this (in powers of two): a weight is then up to
// 2^8, which costs no accuracy, and the weighted sums are rescaled a few times a request instead of every tile.
constexpr float kSlack = 8.0f;

struct SplitArgs {
  const int32_t* lens;
  const int32_t* table;
  int64_t ldt;                       // entries
  int32_t batch, width, n_pages, page;
  int32_t window;                    // 0: all tokens
  int32_t target, least;
  int32_t* pieces;                   // workspace: {first item, number of items} of every request
};

struct Piece {
  int b;
  int begin, end;                    // tokens, begin a multiple of 16 (of 64 without a window)
  int first, len;                    // first token that is seen, tokens of the request
  int item, count;                   // place among all items; pieces of this request
};

struct SplitShared {
  int32_t sum[16], found[4];
};

__device__ __forceinline__ int seen_tokens(const SplitArgs& a, int b, int& first) {
  const int64_t most = (int64_t)a.width * a.page;
  int len = a.lens[b];
  len = len < 0 ? 0 : len > most ? (int)most : len;
  first = a.window > 0 && len > a.window ? len - a.window : 0;
  return len;
}

// Piece `item`; false if there are fewer. T threads, all of them call it.
template <int T, int U>
__device__ __forceinline__ bool find_piece(const SplitArgs& a, int item, SplitShared& sh, Piece& p) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (a.batch + T - 1) / T, from = tid * per, to = min(from + per, a.batch);
  auto units = [&](int b) {
    int first;
    const int len = seen_tokens(a, b, first);
    return (len - (first & ~15) + U - 1) / U;
  };
  int mine = 0;
  for (int b = from; b < to; ++b) mine += units(b);
  int v = lanes_reduce<64>(mine, [](int x, int y) { return x + y; });
  if (lane == 0) sh.sum[wave] = v;
  if (tid == 0) sh.found[0] = -1;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < T / 64; ++w) total += sh.sum[w];
  const int piece = max(a.least, (total + a.target - 1) / a.target);
  auto pieces = [&](int u) { return u <= piece ? 1 : (u + piece - 1) / piece; };
  int count = 0;
  for (int b = from; b < to; ++b) count += pieces(units(b));
  int upto = lanes_before_and_own(count);
  __syncthreads();
  if (lane == 63) sh.sum[wave] = upto;
  __syncthreads();
  for (int w = 0; w < wave; ++w) upto += sh.sum[w];
  if (item < upto && item >= upto - count) {
    int at = upto - count;
    for (int b = from; b < to; ++b) {
      const int n = pieces(units(b));
      if (item < at + n) {
        sh.found[0] = b;
        sh.found[1] = at;
        sh.found[2] = n;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  p.b = __builtin_amdgcn_readfirstlane(sh.found[0]);
  if (p.b < 0) return false;
  const int first_item = __builtin_amdgcn_readfirstlane(sh.found[1]);
  p.count = __builtin_amdgcn_readfirstlane(sh.found[2]);
  p.item = item;
  p.len = seen_tokens(a, p.b, p.first);
  const int origin = p.first & ~15, u = (p.len - origin + U - 1) / U, k = item - first_item;
  // pieces of one request differ by one unit at most
  p.begin = origin + U * (int)((int64_t)u * k / p.count);
  p.end = min(p.len, origin + U * (int)((int64_t)u * (k + 1) / p.count));
  if (k == 0 && tid == 0 && blockIdx.y == 0) {
    a.pieces[2 * p.b] = item;
    a.pieces[2 * p.b + 1] = p.count;
  }
  return true;
}

// v as the sum of two bf16 numbers, within 2^-16 of it: the first is v rounded, this the rest (none beside an infinity).
__device__ __forceinline__ float bf16_rest(float v) {
  const float hi = bf16_f(f_bf16(v));
  return fabsf(hi) < __builtin_inff() ? v - hi : 0.0f;
}

// Sum of a head's pieces: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i, in order. A workgroup has one request and head; its
// waves take every 8th piece, a lane D / 64 columns. Bound by the latency of two rounds of loads. PAIR: the result as two bf16 numbers
// D apart.
struct JoinArgs {
  const int32_t* pieces;
  const float* part;                 // [items][heads][D]
  const float* ml;                   // [items][heads][2]: maximum (base 2), sum of weights
  uint16_t* out;
  float* lse;                        // or null
  int64_t out_b, out_h, lse_b;       // elements
  int32_t heads;
};

constexpr int kJoinWaves = 8;
template <int D, bool PAIR>
__global__ __launch_bounds__(64 * kJoinWaves) void join_kernel(JoinArgs a) {
  constexpr int N = D / 64;
  __shared__ float red[kJoinWaves][D], top[kJoinWaves], sum[kJoinWaves];
  const int b = blockIdx.y, h = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int first = a.pieces[2 * b], n = a.pieces[2 * b + 1];
  if (n < 2) return;                 // written by its only piece
  float m = kNone, l = 0.0f, o[N];
#pragma unroll
  for (int j = 0; j < N; ++j) o[j] = 0.0f;
  constexpr int B = 8;               // loads of eight pieces at once
  for (int i = wave; i < n; i += kJoinWaves * B) {
    float pm[B], pl[B], po[B][N];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int at = i + k * kJoinWaves;
      const int64_t row = (int64_t)(first + (at < n ? at : i)) * a.heads + h;
      pm[k] = at < n ? a.ml[2 * row] : kNone;
      pl[k] = a.ml[2 * row + 1];
#pragma unroll
      for (int j = 0; j < N; ++j) po[k][j] = a.part[row * D + N * lane + j];
    }
    float t = m;
#pragma unroll
    for (int k = 0; k < B; ++k) t = pm[k] > t || pm[k] != pm[k] ? pm[k] : t;
    if (t == kNone) continue;
    const float f = exp2f(m - t);
    l *= f;
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] *= f;
#pragma unroll
    for (int k = 0; k < B; ++k) {
      if (pm[k] == kNone) continue;
      const float g = exp2f(pm[k] - t);
      l = __builtin_fmaf(g, pl[k], l);
#pragma unroll
      for (int j = 0; j < N; ++j) o[j] = __builtin_fmaf(g, po[k][j], o[j]);
    }
    m = t;
  }
  if (lane == 0) {
    top[wave] = m;
    sum[wave] = l;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) red[wave][N * lane + j] = o[j];
  __syncthreads();
  float t = kNone;
#pragma unroll
  for (int w = 0; w < kJoinWaves; ++w) t = top[w] > t || top[w] != top[w] ? top[w] : t;
  float all = 0.0f, g[kJoinWaves];
#pragma unroll
  for (int w = 0; w < kJoinWaves; ++w) {
    g[w] = top[w] == kNone ? 0.0f : exp2f(top[w] - t);
    all = __builtin_fmaf(g[w], sum[w], all);
  }
  const float inv = all == 0.0f ? 0.0f : 1.0f / all;
  for (int d = threadIdx.x; d < D; d += 64 * kJoinWaves) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w)
      if (top[w] != kNone) v = __builtin_fmaf(g[w], red[w][d], v);
    uint16_t* to = a.out + b * a.out_b + h * a.out_h + d;
    to[0] = f_bf16(v * inv);
    if constexpr (PAIR) to[D] = f_bf16(bf16_rest(v * inv));
  }
  if (a.lse && threadIdx.x == 0) a.lse[b * a.lse_b + h] = all == 0.0f ? kNone : (t + log2f(all)) / kLog2E;
}

}  // namespace ops
}  // namespace fg
